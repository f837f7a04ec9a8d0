"""GPU parity of the gated linear recurrence (deltanet_scan_fwd, _bwd, _step) against the
float64 token recurrence in oracle/block_ops.py.

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


def draw(B, T, D, x=BF, g=F, N=None, seed=0, init=True, fused=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    xv, gv = r(B, T, D).to(x), torch.nn.functional.logsigmoid(2 * r(B, T, D) + 3).to(g)
    if fused and x == g:
        both = torch.cat([xv, gv], -1).to(DEV)
        xv, gv = both[..., :D], both[..., D:]
    s0 = r(N or B, D).to(DEV) if init else None
    return xv.to(DEV), gv.to(DEV), s0


def guarded(shape, dtype):
    """A buffer inside a larger one full of a known value, and the check that nothing around
    it was written."""
    n = int(np.prod(shape))
    pad = 256
    big = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)

    def check():
        torch.cuda.synchronize()
        assert (big[:pad] == 7).all() and (big[pad + n:] == 7).all()
    return big[pad:pad + n].view(shape), check


SHAPES = [(1, 1, 1), (2, 1, 7), (2, 3, 5), (1, 16, 64), (3, 17, 66), (2, 63, 130), (2, 130, 33), (1, 513, 64),
          (5, 257, 32), (2, 1000, 192), (1, 4099, 48), (300, 5, 40), (1, 2048, 1026)]
TYPES = [(BF, F), (BF, BF), (F, F)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x,g", TYPES)
def test_forward(shape, x, g):
    B, T, D = shape
    xs, gs, s0 = draw(B, T, D, x, g, seed=T, init=T % 2 == 0, fused=D % 2 == 0)
    out, check = guarded((B, T, D), x)
    fin, check2 = guarded((B, D), F)
    dn.deltanet_scan_fwd(xs, gs, s0, out=out, final_state=fin)
    check(), check2()
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0))
    close(out, h, bh)
    close(fin, final, bf)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x,g", TYPES)
def test_backward(shape, x, g):
    B, T, D = shape
    xs, gs, s0 = draw(B, T, D, x, g, seed=T + 1, init=T % 3 != 0, fused=D % 2 == 0)
    h = dn.deltanet_scan_fwd(xs, gs, s0)[0]
    gen = torch.Generator().manual_seed(T)
    dh = torch.randn((B, T, D), generator=gen).to(DEV, x)
    df = torch.randn((B, D), generator=gen).to(DEV) if T % 2 else None
    dx, c1 = guarded((B, T, D), x)
    dg, c2 = guarded((B, T, D), g)
    ds, c3 = guarded((B, D), F)
    dn.deltanet_scan_bwd(gs, h, dh, s0, None, df, d_x=dx, d_g=dg, d_initial_state=ds)
    c1(), c2(), c3()
    want, bound = ops.scan_bwd(f64(gs), f64(h), f64(dh), f64(s0), None, f64(df))
    for t, w, b in zip((dx, dg, ds), want, bound):
        close(t, w, b)


PACKED = [[0, 1], [0, 0, 1, 1], [0, 5, 5, 6, 40, 40], [0, 0, 0, 64, 128, 129], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 333],
          [0, 700, 701, 1500], list(range(0, 301, 3)) + [900], [0, 513, 513, 2100, 2100]]


@pytest.mark.parametrize("cu", PACKED, ids=lambda c: f"{len(c) - 1}x{c[-1]}")
@pytest.mark.parametrize("x,g,D", [(BF, F, 64), (BF, BF, 35), (F, F, 130)])
def test_packed(cu, x, g, D):
    T, N = cu[-1], len(cu) - 1
    xs, gs, s0 = draw(1, T, D, x, g, N, seed=T, init=N % 2 == 1)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, fin = dn.deltanet_scan_fwd(xs, gs, s0, c)
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0), cu)
    close(out, h, bh)
    close(fin, final, bf)
    gen = torch.Generator().manual_seed(T)
    dh, df = torch.randn((1, T, D), generator=gen).to(DEV, x), torch.randn((N, D), generator=gen).to(DEV)
    ds = torch.empty((N, D), device=DEV)
    got = dn.deltanet_scan_bwd(gs, out, dh, s0, c, df if N % 3 else None, d_initial_state=ds)
    want, bound = ops.scan_bwd(f64(gs), f64(out), f64(dh), f64(s0), cu, f64(df) if N % 3 else None)
    for t, w, b in zip(got, want, bound):
        close(t, w, b)
    assert dn.get_error() == 0


def test_many_short_sequences():
    """More sequences than a warp or a CTA has threads, many without tokens."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 5, size=3000)
    cu = [0] + np.cumsum(lens).tolist()
    xs, gs, s0 = draw(1, cu[-1], 70, BF, F, 3000)
    out, fin = dn.deltanet_scan_fwd(xs, gs, s0, torch.tensor(cu, dtype=torch.int32, device=DEV))
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0), cu)
    close(out, h, bh)
    close(fin, final, bf)


def test_gradients_are_differences():
    """d_x, d_g, d_initial_state of a weighted sum of out and final_state against central
    differences of the library's own forward pass, in fp32 (step 2^-6: the sum's truncation
    error is third order in it, its rounding 2^-24 / 2^-6 of the sum's terms)."""
    B, T, D = 2, 70, 3
    xs, gs, s0 = draw(B, T, D, F, F, seed=9)
    gen = torch.Generator().manual_seed(1)
    wo, wf = torch.randn((B, T, D), generator=gen).to(DEV), torch.randn((B, D), generator=gen).to(DEV)

    def loss(x, g, s):
        out, fin = dn.deltanet_scan_fwd(x, g, s)
        return ((out * wo).double().sum() + (fin * wf).double().sum()).item()

    out, _ = dn.deltanet_scan_fwd(xs, gs, s0)
    grads = dn.deltanet_scan_bwd(gs, out, wo, s0, None, wf)
    for which, at in ((0, (0, 0, 1)), (0, (1, 33, 2)), (0, (1, 69, 0)), (1, (0, 0, 0)), (1, (1, 40, 1)),
                      (1, (0, 69, 2)), (2, (0, 1)), (2, (1, 2))):
        v = [xs.clone(), gs.clone(), s0.clone()]
        e = 2.0 ** -6
        base = v[which][at].item()
        v[which][at] = base + e
        up = loss(*v)
        v[which][at] = base - e
        down = loss(*v)
        want, got = (up - down) / (2 * e), grads[which][at].item()
        # g enters as exp(g): (e^2 / 6) of the gradient's size per token it passes, 1e-4 here
        assert abs(got - want) <= 2e-3 * max(1.0, abs(want)), (which, at, got, want)


@pytest.mark.parametrize("T", [6, 700])
def test_special_decays(T):
    """a = 0 (g = -inf) forgets, a = 1 keeps, a > 1 grows; bf16 gates hold -inf too."""
    for gt in (F, BF):
        xs, gs, s0 = draw(2, T, 66, BF, gt, seed=3)
        gs = gs.clone()
        gs[:, 1::4] = float("-inf")
        gs[:, ::3] = 0.0
        gs[:, 2::5, ::2] = 0.25
        out, fin = dn.deltanet_scan_fwd(xs, gs, s0)
        h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0))
        close(out, h, bh)
        close(fin, final, bf)
        dh = torch.randn((2, T, 66), device=DEV).to(BF)
        got = dn.deltanet_scan_bwd(gs, out, dh, s0)
        want, bound = ops.scan_bwd(f64(gs), f64(out), f64(dh), f64(s0))
        for t, w, b in zip(got, want, bound):
            close(t, w, b)


@pytest.mark.parametrize("x,D", [(BF, 64), (F, 33)])
def test_nan_and_inf_stay_in_their_sequence_and_channel(x, D):
    cu = [0, 40, 41, 200, 200, 900]
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    xs, gs, s0 = draw(1, 900, D, x, F, 5)
    clean = dn.deltanet_scan_fwd(xs, gs, s0, c)
    dh = torch.randn((1, 900, D), device=DEV).to(x)
    clean_b = dn.deltanet_scan_bwd(gs, clean[0], dh, s0, c)
    bad = xs.clone()
    bad[0, 100, 5] = float("nan")
    bad[0, 39, 7] = float("inf")
    bad[0, 199] = float("nan")
    out, fin = dn.deltanet_scan_fwd(bad, gs, s0, c)
    mask = torch.ones((900, D), dtype=torch.bool, device=DEV)
    mask[100:200, 5] = mask[39, 7] = False
    mask[199] = False
    assert torch.equal(out[0][mask], clean[0][0][mask])
    assert torch.isnan(out[0, 100:200, 5]).all() and torch.isinf(out[0, 39, 7]) and torch.isnan(out[0, 199]).all()
    assert torch.equal(fin[[1, 3, 4]], clean[1][[1, 3, 4]])
    bad = dh.clone()
    bad[0, 41] = float("nan")       # first token of sequence 2: nothing before it may see it
    bad[0, 300, 3] = float("inf")
    dx, dg, ds = dn.deltanet_scan_bwd(gs, clean[0], bad, s0, c)
    mask = torch.ones((900, D), dtype=torch.bool, device=DEV)
    mask[41] = False
    mask[200:301, 3] = False
    assert torch.equal(dx[0][mask], clean_b[0][0][mask]) and torch.equal(dg[0][mask], clean_b[1][0][mask])
    assert torch.equal(ds[[0, 1, 3]], clean_b[2][[0, 1, 3]])


def test_invalid_boundaries_are_reported():
    """cu_seqlens that do not start at 0, decrease, or do not end at T (all of them still in
    range of the buffers for the kernels, which clamp)."""
    xs, gs, _ = draw(1, 50, 34, BF, F, init=False)
    for cu in ([1, 20, 50], [0, 30, 20, 50], [0, 20, 49], [0, 20, 51], [0, -5, 50], [0, 2**30, 50]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        out, _ = dn.deltanet_scan_fwd(xs, gs, None, c)
        assert dn.get_error() == _lib.DN_ERR_SEQLENS
        dn.deltanet_scan_bwd(gs, torch.zeros_like(out), xs, None, c)
        assert dn.get_error() == _lib.DN_ERR_SEQLENS
    assert dn.get_error() == 0


def test_no_tokens_no_sequences():
    z = torch.empty((2, 0, 8), device=DEV)
    s0 = torch.randn((2, 8), device=DEV)
    out, fin = dn.deltanet_scan_fwd(z, z, s0)
    assert out.shape == (2, 0, 8) and torch.equal(fin, s0)
    dx, dg, ds = dn.deltanet_scan_bwd(z, z, z, s0, None, s0 * 2)
    assert torch.equal(ds, s0 * 2)
    out, fin = dn.deltanet_scan_fwd(z, z)
    assert not fin.any()
    e = torch.empty((0, 5, 8), device=DEV)
    assert dn.deltanet_scan_fwd(e, e)[1].shape == (0, 8)
    c = torch.zeros(4, dtype=torch.int32, device=DEV)
    p = torch.empty((1, 0, 8), device=DEV)
    s3 = torch.randn((3, 8), device=DEV)
    assert torch.equal(dn.deltanet_scan_fwd(p, p, s3, c)[1], s3)
    assert torch.equal(dn.deltanet_scan_bwd(p, p, p, s3, c, s3)[2], s3)


def test_strided_and_interleaved():
    """Odd pitches, a transposed batch, a broadcast gate and start state, and gradients into
    the two halves of one buffer."""
    B, T, D = 3, 75, 36
    big = torch.randn((T, B, 2 * D + 3), device=DEV).to(BF)
    x = big[:, :, 1:D + 1].transpose(0, 1)
    g = -torch.rand((1, 1, D), device=DEV).expand(B, T, D)
    s0 = torch.randn((1, D), device=DEV).expand(B, D)
    out = torch.zeros((T, B, D + 1), device=DEV, dtype=BF)[..., 1:].transpose(0, 1)
    fin = dn.deltanet_scan_fwd(x, g, s0, out=out)[1]
    h, final, bh, bf = ops.scan(f64(x), f64(g), f64(s0))
    close(out, h, bh)
    close(fin, final, bf)
    gb = g.to(BF)
    both = torch.full((B, T, 2 * D), 9.0, dtype=BF, device=DEV)
    dh = torch.randn((B, T, D), device=DEV).to(BF)
    dn.deltanet_scan_bwd(gb, out, dh, s0, d_x=both[..., :D], d_g=both[..., D:])
    want, bound = ops.scan_bwd(f64(gb), f64(out), f64(dh), f64(s0))
    close(both[..., :D], want[0], bound[0])
    close(both[..., D:], want[1], bound[1])


def test_split_sequence_is_one_sequence():
    """Two calls chained through the state, and the gradients chained back."""
    xs, gs, s0 = draw(2, 401, 66, F, F)
    out, fin = dn.deltanet_scan_fwd(xs, gs, s0)
    o1, f1 = dn.deltanet_scan_fwd(xs[:, :150], gs[:, :150], s0)
    o2, f2 = dn.deltanet_scan_fwd(xs[:, 150:], gs[:, 150:], f1)
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0))
    close(torch.cat([o1, o2], 1), h, 2 * bh)
    close(f2, final, 2 * bf)
    dh, df = torch.randn_like(xs), torch.randn_like(s0)
    _, _, d2 = dn.deltanet_scan_bwd(gs[:, 150:], out[:, 150:], dh[:, 150:], f1, None, df)
    d1 = dn.deltanet_scan_bwd(gs[:, :150], out[:, :150], dh[:, :150], s0, None, d2)[2]
    want, bound = ops.scan_bwd(f64(gs), f64(out), f64(dh), f64(s0), None, f64(df))
    close(d1, want[2], 2 * bound[2])


@pytest.mark.parametrize("N,T,D,M", [(1, 1, 1, 1), (3, 1, 33, 7), (256, 1, 512, 300), (5, 4, 130, 5), (2, 37, 64, 4)])
@pytest.mark.parametrize("x,g", TYPES)
def test_step(N, T, D, M, x, g):
    xs, gs, _ = draw(N, T, D, x, g, fused=True)
    state = torch.randn((M, D), device=DEV)
    slots = torch.randperm(M)[:N].to(torch.int32)
    before = state.clone()
    out, check = guarded((N, T, D), x)
    dn.deltanet_scan_step(xs, gs, state, slots.to(DEV), out=out)
    check()
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(before)[slots.numpy()])
    close(out, h, bh)
    want, bound = f64(before), np.zeros(before.shape)
    want[slots.numpy()], bound[slots.numpy()] = final, bf
    close(state, want, bound)
    others = torch.ones(M, dtype=torch.bool)
    others[slots.long()] = False
    assert torch.equal(state[others.to(DEV)], before[others.to(DEV)])
    if N == M:
        state2 = before.clone()
        out2 = dn.deltanet_scan_step(xs, gs, state2)
        h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(before))
        close(out2, h, bh)
        close(state2, final, bf)
    assert dn.get_error() == 0


def test_step_padding_and_bad_slots():
    xs, gs, _ = draw(6, 2, 300, BF, F)
    state = torch.randn((4, 300), device=DEV)
    before = state.clone()
    ok = torch.tensor([2, -1, 0, -1, 3, 1], dtype=torch.int32, device=DEV)
    out = dn.deltanet_scan_step(xs, gs, state, ok)
    assert dn.get_error() == 0 and not out[[1, 3]].any() and out[[0, 2, 4, 5]].any(-1).all()
    for bad in ([2, 2, 0, -1, 3, 1], [2, -2, 0, -1, 3, 1], [2, 4, 0, -1, 3, 1], [2, 2**31 - 1, 0, -1, 3, 1]):
        st = before.clone()
        o = dn.deltanet_scan_step(xs, gs, st, torch.tensor(bad, dtype=torch.int32, device=DEV))
        assert dn.get_error() == _lib.DN_ERR_SLOTS
        assert torch.equal(st, state) and torch.equal(o, out)
    assert dn.get_error() == 0


def test_captured_calls_and_streams():
    """Graphs of a forward, backward and step call replay on new inputs, two of them on two
    streams at once; a call given a stream runs there."""
    side = torch.cuda.Stream()
    cases = []
    for seed in (0, 1):
        xs, gs, s0 = draw(1, 700, 130, BF, F, 3, seed=seed)
        c = torch.tensor([0, 300, 300, 700], dtype=torch.int32, device=DEV)
        cases.append((xs, gs, s0, c, torch.randn((1, 700, 130), device=DEV).to(BF)))

    def chain(xs, gs, s0, c, dh):
        out, fin = dn.deltanet_scan_fwd(xs, gs, s0, c)
        return [out, fin, *dn.deltanet_scan_bwd(gs, out, dh, s0, c, fin)]

    want = [chain(*k) for k in cases]
    torch.cuda.synchronize()
    graphs, outs, ins = [], [], []
    for k in cases:
        st = [t.clone() for t in k]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            chain(*st)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            o = chain(*st)
        graphs.append(gr), outs.append(o), ins.append(st)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for swap in (0, 1):
        for i in (0, 1):
            for t, s in zip(ins[i], cases[i ^ swap]):
                t.copy_(s)
        torch.cuda.synchronize()
        for _ in range(3):
            for i in (0, 1):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            for a, b in zip(outs[i], want[i ^ swap]):
                assert torch.equal(a, b)
    xs, gs, s0, c, dh = cases[0]
    out, fin = dn.deltanet_scan_fwd(xs, gs, s0, c, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(fin, want[0][1])
    assert dn.get_error() == 0 and dn.get_error(side) == 0


def test_capture_before_the_first_call_on_a_stream_is_refused_softly():
    """Packed input needs the stream's error word; inside a capture that cannot be made, and
    the capture goes on without the call."""
    xs, gs, s0 = draw(1, 40, 32, BF, F, 1)
    c = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream(priority=-1)
    t = torch.zeros(1, device=DEV)
    gr = torch.cuda.CUDAGraph()
    seen = []
    torch.cuda.synchronize()
    with torch.cuda.graph(gr, stream=s):
        try:
            dn.deltanet_scan_fwd(xs, gs, s0, c)
        except dn.DeltaNetError as e:
            seen.append(e.status)
        out, _ = dn.deltanet_scan_fwd(xs, gs, s0)        # dense: needs none
        t += 1
    gr.replay()
    torch.cuda.synchronize()
    assert t.item() == 1
    if seen:      # torch hands out pooled streams: this one may have had a call before
        assert seen == [_lib.DN_ERR_WORKSPACE]
    assert torch.equal(out, dn.deltanet_scan_fwd(xs, gs, s0)[0])


@pytest.mark.parametrize("B,T,D", [(1, 32768, 2048), (8, 4096, 2048), (1, 20000, 514)])
def test_backward_under_load(B, T, D):
    """Every d_g of a large call is a h_{t-1} times its d_x (which is rounded, and so is d_g:
    2^-8 each): nothing is read before it has arrived, the first tokens of a row included,
    which are worked on last."""
    xs, gs, s0 = draw(1, 64, D, BF, F)
    h = torch.randn((B, T, D), device=DEV).to(BF)
    dh = torch.randn((B, T, D), device=DEV).to(BF)
    g = gs.repeat(B, T // 64 + 1, 1)[:, :T].contiguous()
    s0 = torch.randn((B, D), device=DEV)
    for _ in range(3):
        dx, dg, _ = dn.deltanet_scan_bwd(g, h, dh, s0)
        before = torch.cat([s0[:, None], h[:, :-1].float()], 1)
        want = g.exp() * before * dx.float()
        assert ((dg - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()
        del before, want, dx, dg


def test_same_call_same_bits():
    xs, gs, s0 = draw(2, 3000, 260, BF, F)
    a, b = dn.deltanet_scan_fwd(xs, gs, s0), dn.deltanet_scan_fwd(xs, gs, s0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p, q = dn.deltanet_scan_bwd(gs, a[0], xs, s0), dn.deltanet_scan_bwd(gs, a[0], xs, s0)
    assert all(torch.equal(u, v) for u, v in zip(p, q))


@pytest.mark.slow
def test_offsets_past_31_bits():
    """A tensor of more than 2^31 elements: the last channels and tokens agree with the same
    rows computed alone."""
    T, D = 1 << 20, 2064
    x = torch.randn((1, T, D), device=DEV, dtype=BF)
    g = torch.full((1, 1, D), -0.05, device=DEV).expand(1, T, D)
    out, fin = dn.deltanet_scan_fwd(x, g)
    tail = slice(T - 4096, T)
    # after 4096 tokens at a = e^-0.05 the start state's weight is e^-204: the tail stands alone
    ref, rfin = dn.deltanet_scan_fwd(x[:, tail], g[:, tail])
    h, final, bh, bf = ops.scan(f64(x[:, tail, -40:]), f64(g[:, tail, -40:]))
    close(ref[..., -40:], h, bh)
    late = slice(T - 2048, T)
    close(out[:, late, -40:], h[:, 2048:], bh[:, 2048:])
    close(fin[:, -40:], final, bf)
