"""GPU parity of deltanet_step (the delta-rule recurrences for a few tokens on a cache of
states) against the float64 definition in oracle/block_ops.py, and against the chunkwise
forward pass.

Tolerance: the oracle's bound on 32-bit roundings, element by element, plus half a step
of the output's type.
"""
import numpy as np
import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn
from deltanet_chunkwise_delta_b200 import _lib
from oracle import block_ops as ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(t, want, bound):
    got = f64(t)
    tol = bound + HALF[t.dtype] * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


def draw(N, T, H, dk, dv, x=BF, rule="gdn", nh=1, M=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)
    decay = lambda *s: torch.nn.functional.logsigmoid(r(*s) + 3).to(DEV)
    g = {"delta": lambda: None, "gdn": lambda: decay(N, T, H), "kda": lambda: decay(N, T, H, dk)}[rule]()
    M = M or N
    return dict(q=unit(r(N, T, H, dk)).to(DEV, x), k=unit(r(N, T * nh, H, dk)).to(DEV, x),
                v=r(N, T * nh, H, dv).to(DEV, x), beta=torch.sigmoid(r(N, T * nh, H)).to(DEV),
                state=(0.3 * r(M, H, dk, dv)).to(DEV), g=g, n_h=nh,
                slot_idx=torch.randperm(M, generator=gen)[:N].to(torch.int32).to(DEV))


def run(c, **kw):
    return dn.deltanet_step(**{**c, **kw})


def want(c, before, slots="slot_idx"):
    s = c[slots].cpu().tolist() if c.get(slots) is not None else None
    return ops.delta_step(*(f64(c[k]) for k in ("q", "k", "v", "beta")), f64(before), f64(c["g"]), c["n_h"], s)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("x", [BF, F])
@pytest.mark.parametrize("rule,nh", [("delta", 1), ("gdn", 1), ("kda", 1), ("gdn", 3), ("delta", 2), ("kda", 2)])
def test_parity(dk, dv, x, rule, nh):
    for N, T, H, M in ((1, 1, 1, 1), (3, 1, 5, 4), (2, 6, 2, 9)):
        c = draw(N, T, H, dk, dv, x, rule, nh, M, seed=N + T)
        before = c["state"].clone()
        out = run(c)
        (o, s), (bo, bs) = want(c, before)
        close(out, o, bo)
        close(c["state"], s, bs)
        rest = torch.ones(M, dtype=torch.bool, device=DEV)
        rest[c["slot_idx"].long()] = False
        assert torch.equal(c["state"][rest], before[rest])
    assert dn.get_error() == 0


def test_rows_in_order_without_slots_and_large_batches():
    c = draw(300, 1, 3, 64, 64, BF, "gdn")
    c["slot_idx"] = None
    before = c["state"].clone()
    out = run(c)
    (o, s), (bo, bs) = want(c, before)
    close(out, o, bo)
    close(c["state"], s, bs)


@pytest.mark.parametrize("rule,fn", [("delta", "deltanet_fwd"), ("gdn", "gated_deltanet_fwd"), ("kda", "kda_fwd")])
def test_steps_continue_the_chunkwise_forward(rule, fn):
    """130 tokens in one chunkwise call == 120 in one, then 7 + 1 + 1 + 1 by steps on its
    final state (bf16: the forward pass's own bar, 1e-2 of the largest value)."""
    c = draw(2, 130, 4, 128, 128, BF, rule)
    args = lambda a, b: [c[k][:, a:b] for k in ("q", "k", "v", "beta")] + ([c["g"][:, a:b]] if rule != "delta" else [])
    full, ffin = getattr(dn, fn)(*args(0, 130))
    head, state = getattr(dn, fn)(*args(0, 120))
    outs = [head]
    for a, b in ((120, 127), (127, 128), (128, 129), (129, 130)):
        g = c["g"][:, a:b] if rule != "delta" else None
        outs.append(dn.deltanet_step(*args(a, b)[:4], state, g))
    got = torch.cat(outs, 1)
    assert dn.get_error() == 0
    rel = lambda a, b: ((a.float() - b.float()).abs().max() / b.float().abs().max()).item()
    assert rel(got, full) <= 1e-2 and rel(state, ffin) <= 1e-2


def test_one_token_at_a_time_is_all_at_once():
    """The same tokens in one call or in several: the same arithmetic, the same bits."""
    c = draw(3, 5, 2, 128, 64, F, "kda", 1, 3)
    s1, s2 = c["state"].clone(), c["state"].clone()
    whole = run(c, state=s1)
    parts = [run(c, state=s2, **{k: c[k][:, t:t + 1] for k in ("q", "k", "v", "beta", "g")}) for t in range(5)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s1, s2)


def test_padding_and_bad_slots():
    c = draw(6, 2, 2, 64, 128, BF, "gdn", 1, 4)
    before = c["state"].clone()
    c["slot_idx"] = torch.tensor([2, -1, 0, -1, 3, 1], dtype=torch.int32, device=DEV)
    out = run(c)
    assert dn.get_error() == 0 and not out[[1, 3]].any()
    (o, s), (bo, bs) = want(c, before)
    close(out, o, bo)
    close(c["state"], s, bs)
    for bad in ([2, 2, 0, 2, 3, 1], [2, -2, 0, -1, 3, 1], [2, 4, 0, -1, 3, 1], [2, -2**31, 0, 2**31 - 1, 3, 1]):
        st = before.clone()
        idx = torch.tensor(bad, dtype=torch.int32, device=DEV)
        o = run(c, state=st, slot_idx=idx)
        assert dn.get_error() == _lib.DN_ERR_SLOTS
        assert torch.equal(st, c["state"]) and torch.equal(o, out)
    # all padding: nothing happens
    st = before.clone()
    o = run(c, state=st, slot_idx=torch.full((6,), -1, dtype=torch.int32, device=DEV))
    assert torch.equal(st, before) and not o.any() and dn.get_error() == 0


def test_nan_in_unnamed_rows_and_padding_requests():
    """What padding requests and unnamed rows hold reaches no result."""
    c = draw(4, 1, 2, 64, 64, BF, "kda", 1, 6)
    c["slot_idx"] = torch.tensor([5, -1, 2, -1], dtype=torch.int32, device=DEV)
    clean_state = c["state"].clone()
    clean = run(c, state=clean_state)
    for k in ("q", "k", "v", "beta", "g"):
        c[k][[1, 3]] = float("nan")
    c["state"][[0, 1, 3, 4]] = float("nan")
    out = run(c)
    assert torch.equal(out, clean) and torch.equal(c["state"][[2, 5]], clean_state[[2, 5]])
    assert torch.isnan(c["state"][[0, 1, 3, 4]]).all()


def test_zero_decay_drops_what_the_state_held():
    """a = 0 (g = -inf): finite states are forgotten."""
    c = draw(2, 1, 2, 64, 64, F, "gdn")
    c["g"][0] = float("-inf")
    before = c["state"].clone()
    out = run(c)
    z = before.clone()
    z[c["slot_idx"][0].long()] = 0
    g0 = c["g"].clone()
    g0[0] = 0
    s2 = z.clone()
    out2 = run(c, state=s2, g=g0)
    assert torch.equal(out, out2) and torch.equal(c["state"], s2)


def test_strides():
    """q, k and v as views of one fused projection's output, a cache of layers [M, L, H, ..]."""
    c = draw(3, 2, 2, 64, 64, BF, "gdn", 1, 5)
    fused = torch.cat([c["q"], c["k"], c["v"]], -1)
    v = dict(q=fused[..., :64], k=fused[..., 64:128], v=fused[..., 128:])
    cache = torch.randn((5, 3, 2, 64, 64), device=DEV)
    cache[:, 1] = c["state"]
    keep = cache.clone()
    out = run(c)
    out2 = run(c, state=cache[:, 1], **v)
    assert torch.equal(out, out2) and torch.equal(cache[:, 1], c["state"])
    assert torch.equal(cache[:, [0, 2]], keep[:, [0, 2]])


def test_state_rows_past_31_bits():
    """A cache of more than 2^31 elements (and 2^33 bytes)."""
    M, H = 8300, 16
    cache = torch.zeros((M, H, 128, 128), device=DEV)
    c = draw(3, 1, H, 128, 128, BF, "gdn", 1, 3)
    rows = torch.tensor([M - 1, 8195, 0], device=DEV)
    cache[rows] = c["state"]
    c["slot_idx"] = torch.arange(3, dtype=torch.int32, device=DEV)
    out = run(c)
    out2 = run(c, state=cache, slot_idx=rows.to(torch.int32))
    assert torch.equal(out, out2) and torch.equal(cache[rows], c["state"])
    assert not cache[1:8195].any() and not cache[8196:M - 1].any()


def test_no_tokens_or_requests():
    c = draw(2, 0, 2, 64, 64, BF, "gdn", 1, 3)
    before = c["state"].clone()
    assert run(c).shape == (2, 0, 2, 64) and torch.equal(c["state"], before)
    c = draw(0, 1, 2, 64, 64, BF, "delta", 1, 3)
    assert run(c).shape == (0, 1, 2, 64)


def test_captured_steps_replay_on_a_growing_state():
    """Decoding as it is captured: one graph per call, replayed with the inputs and slots of
    each step copied in; two graphs from one stream replay side by side on their own caches."""
    side = torch.cuda.Stream()
    cs = [draw(4, 1, 2, 128, 128, BF, "gdn", 1, 8, seed=s) for s in (0, 1)]
    steps = [[draw(4, 1, 2, 128, 128, BF, "gdn", 1, 8, seed=10 * s + t) for t in range(4)] for s in (0, 1)]
    ref_state = [c["state"].clone() for c in cs]
    ref = [[run(x, state=ref_state[i]) for x in steps[i]] for i in (0, 1)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cs:
        keep = c["state"].clone()
        with torch.cuda.stream(side):
            run(c)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(run(c))
        graphs.append(gr)
        c["state"].copy_(keep)
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for t in range(4):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                for k in ("q", "k", "v", "beta", "g", "slot_idx"):
                    cs[i][k].copy_(steps[i][t][k])
                graphs[i].replay()
                got[i].append(outs[i].clone())
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(got[i], ref[i]))
        assert torch.equal(cs[i]["state"], ref_state[i])
    assert dn.get_error(side) == 0
