"""The gated linear recurrence where products of decays over a run of tokens pass what fp32
holds, though every h does not: growing gates, tiny start states.

Tolerance: the oracle's bound on 32-bit roundings with the one rounding that it leaves out.  The
logarithm of a run's decays is a sum of up to 84 of them; each of its additions, 1.25 a token
with those over the runs, rounds by U = 2^-24 of the partial sum, P at most.  A token's decay
then carries (6 + 2 |g| + 1.25 P) U where the oracle takes (6 + 2 |g|) U, so its bound times
1 + 1.25 P / 6 holds.

Where h falls below 2^-126, a number rounds by up to 2^-150 whatever its size, and later decays
multiply that: four such roundings a token (a run's two steps, the token's, the sum's), run
through the recurrence themselves, are added.  bf16 rounds by 2^-134 there.
"""
import numpy as np
import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn
from oracle import block_ops as ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}
TYPES = [(F, F), (BF, F), (BF, BF)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def factor(g):
    """1 + 1.25 P / 6 with P the largest |sum of g| over up to 84 tokens in a row."""
    s = np.concatenate([np.zeros_like(g[:, :1]), np.cumsum(g, axis=1)], axis=1)
    P = max(np.abs(s[:, n:] - s[:, :-n]).max() for n in range(1, min(84, g.shape[1]) + 1))
    return 1 + 1.25 * P / 6


def close(t, want, bound, tiny):
    got = f64(t)
    tol = bound + HALF[t.dtype] * np.abs(want) + tiny
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


SHAPES = [(1, 2048, 64, None), (2, 100, 64, None), (2, 150, 33, None), (1, 1500, 35, None),
          (1, 2048, 66, [0, 500, 500, 1400, 2048]), (1, 120, 64, [0, 70, 120])]


@pytest.mark.parametrize("B,T,D,cu", SHAPES, ids=lambda v: None if isinstance(v, list) else str(v))
@pytest.mark.parametrize("x,g", TYPES)
def test_runs_that_grow(B, T, D, cu, x, g):
    """Decays of about e^1.7 for 56 tokens, then of e^-1.7, and so on: the product over 56 tokens
    reaches e^95 (fp32 ends at e^88.7), h stays between 1e-27 and 1e19, but in sequences that do
    not start with the rise, where it falls below fp32's normal numbers."""
    gen = torch.Generator().manual_seed(T + D)
    r = lambda *s: torch.randn(s, generator=gen)
    N = len(cu) - 1 if cu else B
    sign = 1.0 - 2.0 * (torch.arange(T) // 56 % 2)
    gs = (1.7 * sign[None, :, None] + 0.05 * r(B, T, D)).to(DEV, g)
    s0 = (1e-25 * r(N, D)).to(DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV) if cu else None
    k = factor(f64(gs))
    sub = np.full((B, T, D), 2.0 ** -148), np.full((N, D), 2.0 ** -148)
    eh, ef, _, _ = ops.scan(sub[0], f64(gs), sub[1], cu)
    for xs in (torch.zeros((B, T, D)), 1e-25 * r(B, T, D)):
        xs = xs.to(DEV, x)
        out, fin = dn.deltanet_scan_fwd(xs, gs, s0, c)
        h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0), cu)
        close(out, h, k * bh + eh, 2.0 ** -134)
        close(fin, final, k * bf + ef, 0.0)
    dh, df = (1e-25 * r(B, T, D)).to(DEV, x), (1e-25 * r(N, D)).to(DEV)
    got = dn.deltanet_scan_bwd(gs, out, dh, s0, c, df)
    want, bound = ops.scan_bwd(f64(gs), f64(out), f64(dh), f64(s0), cu, f64(df))
    few, _ = ops.scan_bwd(f64(gs), np.abs(f64(out)), sub[0], np.abs(f64(s0)), cu, sub[1])
    for t, w, b, e in zip(got, want, bound, few):
        close(t, w, k * b + e, 1e-37)
    assert dn.get_error() == 0


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("x,g", TYPES)
def test_a_subnormal_state_that_grows_past_one(x, g, split):
    """Decays of e^184.8 over one run (a warp's, or a CTA's of a cluster) on a start state of
    2^-146: the product passes 2^254, where h is 2^120 at most."""
    run = (8 if x == BF else 4) if not split else 84 if x == BF else 56
    T = 12 * run if not split else 4 * run
    sign = 1.0 - 2.0 * (torch.arange(T) // run % 2)
    gs = (184.8 / run * sign)[None, :, None].expand(1, T, 64).to(DEV, g)
    xs, s0 = torch.zeros((1, T, 64), dtype=x, device=DEV), torch.full((1, 64), 2.0 ** -146, device=DEV)
    out, fin = dn.deltanet_scan_fwd(xs, gs, s0)
    h, final, bh, bf = ops.scan(f64(xs), f64(gs), f64(s0))
    k = factor(f64(gs))
    sub = np.full((1, T, 64), 2.0 ** -148)
    eh = ops.scan(sub, f64(gs))[0]
    # the first rise: in the fall after it h rounds to 0, and nothing is left to grow
    close(out[:, :run], h[:, :run], k * bh[:, :run] + eh[:, :run], 2.0 ** -134)
    assert np.isfinite(h).all() and h.max() > 2.0 ** 118
    dh, df = torch.zeros_like(xs), torch.full((1, 64), 2.0 ** -146, device=DEV)
    dx = dn.deltanet_scan_bwd(gs.flip(1), xs, dh, s0, None, df)[0]
    want, bound = ops.scan_bwd(f64(gs.flip(1)), f64(xs), f64(dh), f64(s0), None, f64(df))
    few = ops.scan_bwd(f64(gs.flip(1)), f64(xs), sub)[0][0]
    close(dx[:, T - run:], want[0][:, T - run:], k * bound[0][:, T - run:] + few[:, T - run:], 2.0 ** -134)


@pytest.mark.slow
def test_the_widest_rows():
    """The largest D that is taken, for the step and (fewer tokens than that fill the GPU) the
    walkers; the last channels against the same channels alone."""
    D = 2 ** 31 - 16385
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.zeros((1, 1, D), dtype=BF, device=DEV)
    g = torch.full((1, 1, 1), -0.5, dtype=BF, device=DEV).expand(1, 1, D).contiguous()
    state = torch.ones((1, D), device=DEV)
    tail = slice(D - 5000, D)
    for t in (x, state):
        t[..., tail].copy_(torch.randn((5000,), generator=gen, device=DEV))
    ref = state[:, tail].clone()
    want = dn.deltanet_scan_step(x[..., tail], g[..., tail], ref)
    got = dn.deltanet_scan_step(x, g, state)
    assert torch.equal(got[..., tail], want) and torch.equal(state[:, tail], ref)
    assert (state[:, :5] == state[0, 0]).all() and torch.equal(state[0, D // 2:D // 2 + 5], state[0, :5])
    del got
    out, fin = dn.deltanet_scan_fwd(x, g, state)
    want, wfin = dn.deltanet_scan_fwd(x[..., tail], g[..., tail], state[:, tail])
    assert torch.equal(out[..., tail], want) and torch.equal(fin[:, tail], wfin)
    assert (out[0, 0, :5] == out[0, 0, D // 2]).all()
    dx, dg, ds = dn.deltanet_scan_bwd(g, out, x, state)
    want = dn.deltanet_scan_bwd(g[..., tail], out[..., tail], x[..., tail], state[:, tail])
    for a, b in zip((dx, dg, ds), want):
        assert torch.equal(a[..., tail], b)
