"""GPU parity of the norms around a block (deltanet_norm_fwd, deltanet_norm_bwd) against the
float64 definition in oracle/block_ops.py.

Tolerance: the oracle's bound on 32-bit roundings, element by element, plus half a step
of the output's type.
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
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(t, want, bound, what=""):
    got = f64(t)
    tol = bound + HALF[t.dtype] * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


PARTS = ["w", "z", "r", "wz", "rn", "rs", "wzr", "rsn", "wzrsn"]


def draw(shape, parts, y=BF, r=BF, wt=F, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)
    d = shape[-1]
    has_out = "r" not in parts or "n" in parts
    return dict(y=(2 * n(*shape)).to(DEV, y), w=(1 + 0.2 * n(d)).to(DEV, wt) if "w" in parts else None,
                z=(2 * n(*shape)).to(DEV, y) if "z" in parts else None,
                r=n(*shape).to(DEV, r) if "r" in parts else None,
                s=(0.5 + 0.2 * n(d)).to(DEV, wt) if "s" in parts else None,
                nw=(1 + 0.2 * n(d)).to(DEV, wt) if "n" in parts else None,
                dout=n(*shape).to(DEV, y) if has_out else None,
                dr=n(*shape).to(DEV, r) if "r" in parts else None)


def forward(c, act="silu", **kw):
    return dn.deltanet_norm_fwd(c["y"], c["w"], c["z"], c["r"], c["s"], c["nw"], activation=act, eps=EPS, **kw)


def backward(c, act="silu", **kw):
    return dn.deltanet_norm_bwd(c["y"], c["dout"], c["w"], c["z"], c["r"], c["s"], c["nw"], c["dr"],
                                activation=act, eps=EPS, **kw)


def check(c, act="silu", fwd=None, bwd=None):
    v = {k: f64(t) for k, t in c.items()}
    a = (v["w"], v["z"], act, v["r"], v["s"], v["nw"])
    (out, rp), (bo, br) = ops.norm(v["y"], *a, EPS)
    got = fwd or forward(c, act)
    for t, w, b, n in ((got[0], out, bo, "out"), (got[1], rp, br, "residual_out")):
        assert (t is None) == (w is None)
        if t is not None:
            close(t, w, b, n)
    want, bound = ops.norm_bwd(v["y"], v["dout"], *a, v["dr"], EPS)
    gr = bwd or backward(c, act)
    got = dict(y=gr.d_y, weight=gr.d_weight, gate=gr.d_gate, residual=gr.d_residual, scale=gr.d_scale,
               next=gr.d_next_weight)
    assert {k for k, t in got.items() if t is not None} == set(want)
    for k in want:
        close(got[k], want[k], bound[k], k)


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("y,r,wt", [(BF, BF, F), (BF, F, BF), (F, F, F)])
def test_parity(parts, y, r, wt):
    for i, shape in enumerate([(2, 3, 5, 128), (3, 7, 264), (1, 1), (5, 33), (2, 2, 1024), (3, 2, 2048)]):
        check(draw(shape, parts, y, r, wt, seed=i), "sigmoid" if i % 2 else "silu")


@pytest.mark.parametrize("d", [1, 2, 7, 31, 32, 63, 64, 80, 96, 127, 128, 160, 255, 256, 511, 512, 513, 768, 1000, 1111,
                               1280, 1536, 2560, 4095, 4096, 5120, 8192, 8200, 12289, 16384])
@pytest.mark.parametrize("y,r", [(BF, BF), (F, F)])
def test_row_lengths(d, y, r):
    rows = 3 if d > 4096 else 37
    check(draw((rows, d), "wzrsn", y, r, seed=d))
    check(draw((rows, d), "wz", y, r, seed=d), "sigmoid")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 31, 147, 148, 149, 295, 297, 593, 1185, 4737])
def test_row_counts(rows):
    check(draw((rows, 64), "wz", seed=rows))
    check(draw((rows, 200), "wzrsn", BF, F, seed=rows))


def test_many_heads():
    check(draw((2, 601, 16, 128), "wz"))


def test_strides_broadcasts_and_interleaved_outputs():
    """Odd pitches, a gate beside y in one buffer, a transposed batch, a residual shared by all
    rows, outputs side by side in one buffer."""
    c = draw((3, 5, 2, 64), "wz")
    both = torch.cat([c["y"], c["z"]], -1)
    v = {**c, "y": both[..., :64], "z": both[..., 64:], "dout": c["dout"].transpose(0, 1).contiguous().transpose(0, 1)}
    out = torch.full((3, 5, 2, 131), 5.0, dtype=BF, device=DEV)
    grads = torch.full((3, 5, 2, 128), 5.0, dtype=BF, device=DEV)
    check(v, fwd=forward(v, out=out[..., 1:65]),
          bwd=backward(v, d_y=grads[..., :64], d_gate=grads[..., 64:]))
    assert (out[..., 0] == 5).all() and (out[..., 65:] == 5).all()
    c = draw((4, 6, 250), "wzrsn", BF, F)
    wide = torch.zeros((4, 6, 253), dtype=BF, device=DEV)
    wide[..., 3:] = c["y"]
    v = {**c, "y": wide[..., 3:], "r": c["r"][:1, :1].expand(4, 6, 250)}
    check(v)


def test_guards():
    """Nothing around the outputs is written, at odd sizes and the largest row."""
    for shape in ((7, 33), (5, 1111), (2, 16384), (9, 128)):
        c = draw(shape, "wzrsn", BF, BF)
        n = shape[0] * shape[1]
        bufs = [torch.full((n + 128,), 5.0, dtype=BF, device=DEV) for _ in range(5)]
        v = [b[64:64 + n].view(shape) for b in bufs]
        fwd = forward(c, out=v[0], residual_out=v[1])
        bwd = backward(c, d_y=v[2], d_gate=v[3], d_residual=v[4])
        check(c, fwd=fwd, bwd=bwd)
        for b in bufs:
            assert (b[:64] == 5).all() and (b[64 + n:] == 5).all()


def test_l2_norm_of_q_and_k():
    """weight d^-1/2 and eps / d: x / sqrt(sum x^2 + eps), the normalisation of q and k."""
    x = torch.randn((2, 9, 3, 128), device=DEV)
    w = torch.full((128,), 128 ** -0.5, device=DEV)
    out, _ = dn.deltanet_norm_fwd(x, w, eps=1e-6 / 128)
    ref = f64(x) / np.sqrt((f64(x) ** 2).sum(-1, keepdims=True) + 1e-6)
    close(out, ref, 40 * ops.U * np.abs(ref))        # w rounded once, its square within the root


def test_gradients_are_differences():
    """The library's gradients against central differences of its own forward pass in fp32
    (step 2^-7; the loss sums 2 x 3 x 40 terms of size 1 in 64 bits, each off by about 2^-22,
    over 2^-6: below 1e-3)."""
    c = draw((2, 3, 40), "wzrsn", F, F, seed=5)
    for act in ("silu", "sigmoid"):
        gr = backward(c, act)

        def loss(k):
            out, rp = forward(k, act)
            return ((out * c["dout"]).double().sum() + (rp * c["dr"]).double().sum()).item()

        for name, grad in (("y", gr.d_y), ("w", gr.d_weight), ("z", gr.d_gate), ("r", gr.d_residual),
                           ("s", gr.d_scale), ("nw", gr.d_next_weight)):
            for at in ((0,) * (c[name].dim() - 1) + (3,), tuple(n - 1 for n in c[name].shape)):
                e, v = 2.0 ** -7, dict(c)
                v[name] = c[name].clone()
                v[name][at] += e
                up = loss(v)
                v[name][at] -= 2 * e
                diff, got = (up - loss(v)) / (2 * e), grad[at].item()
                assert abs(got - diff) <= 2e-3 * max(1.0, abs(diff)), (act, name, at, got, diff)


def test_missing_residual_gradient_is_zero():
    c = draw((5, 96), "wzrsn")
    c["dr"] = None
    a = backward(c)
    c["dr"] = torch.zeros((5, 96), dtype=BF, device=DEV)
    b = backward(c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_nan_and_inf_stay_in_their_row():
    """A row with NaN or infinities touches no other row; the parameters' sums take it in."""
    for d in (128, 300, 2048):
        c = draw((9, d), "wzrsn")
        a, ga = forward(c), backward(c)
        v = {**c, "y": c["y"].clone(), "z": c["z"].clone(), "dout": c["dout"].clone()}
        v["y"][2, 1] = float("nan")
        v["z"][4, 0] = float("inf")
        v["dout"][6, d - 1] = float("-inf")
        b, gb = forward(v), backward(v)
        for rows in ([0, 1, 3, 5, 7, 8],):
            for x, y in ((a[0], b[0]), (a[1], b[1]), (ga.d_y, gb.d_y), (ga.d_gate, gb.d_gate),
                         (ga.d_residual, gb.d_residual)):
                assert torch.equal(x[rows], y[rows])
        assert torch.isnan(b[0][2]).all() and not torch.isfinite(gb.d_weight).all()


def test_infinite_weight_with_fewer_rows_than_a_cta_takes():
    """y1 is infinite in one column, and so is that column of d_scale; the places of rows that
    a CTA has room for and the call does not have add nothing (0 times inf would be NaN)."""
    for d in (64, 65, 128, 256):
        c = draw((3, d), "wrs")
        c["y"], c["dr"] = c["y"].abs() + 0.5, c["dr"].abs() + 0.5
        base = backward(c)
        c["w"][5] = float("inf")
        gr = backward(c)
        assert gr.d_scale[5] == float("inf")
        rest = [i for i in range(d) if i != 5]
        assert torch.equal(gr.d_scale[rest], base.d_scale[rest])
        assert torch.equal(gr.d_residual, base.d_residual)


def test_extreme_gates_and_zero_rows():
    """Gates far out (the sigmoid is 0 or 1 there), rows of zeros (rstd is eps^-1/2)."""
    c = draw((6, 64), "wz")
    c["z"][0], c["z"][1], c["z"][2] = 200.0, -200.0, -87.5
    c["y"][3] = 0
    for act in ("silu", "sigmoid"):
        out, _ = forward(c, act)
        gr = backward(c, act)
        assert torch.isfinite(out).all() and all(torch.isfinite(t).all() for t in gr if t is not None)
        assert not out[1].any() and not out[3].any()
        assert not gr.d_gate[0].any() if act == "sigmoid" else gr.d_gate[0].any()


def test_no_rows():
    c = draw((0, 5, 64), "wzrsn")
    out, rp = forward(c)
    gr = backward(c)
    assert out.shape == rp.shape == gr.d_y.shape == (0, 5, 64)
    assert not gr.d_weight.any() and not gr.d_scale.any() and not gr.d_next_weight.any()


def test_same_call_same_bits():
    c = draw((1200, 192), "wzrsn")
    a, b = backward(c), backward(c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_calls_and_streams():
    """Forward and backward in a graph, two graphs captured on one stream replayed side by side
    (each has its own workspace), and calls on a stream that is not the current one."""
    side = torch.cuda.Stream()
    cs = [draw((700, 512), "wzrsn", seed=s) for s in (0, 1)]
    want = [(*forward(c), *backward(c)) for c in cs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append((*forward(c), *backward(c)))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    o = (*forward(cs[0], stream=side), *backward(cs[0], stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want[0]))


@pytest.mark.slow
def test_offsets_past_31_bits():
    """More than 2^31 elements: the last rows agree with themselves alone."""
    rows, d = (1 << 20) + 3, 2056
    y = torch.randn((rows, d), device=DEV, dtype=BF)
    w = torch.ones(d, device=DEV)
    out, _ = dn.deltanet_norm_fwd(y, w)
    tail, _ = dn.deltanet_norm_fwd(y[-5:], w)
    assert torch.equal(out[-5:], tail)
    gr = dn.deltanet_norm_bwd(y, y, w)
    assert torch.equal(gr.d_y[-5:], dn.deltanet_norm_bwd(y[-5:], y[-5:], w).d_y)
