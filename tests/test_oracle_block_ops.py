"""Pins of the float64 definitions in oracle/block_ops.py: closed forms, the token
recurrence of oracle/deltanet_oracle.c, and gradients against central differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block_ops as ops


def test_scan_closed_form():
    """h_t = sum_s exp(g_{s+1} + .. + g_t) x_s + exp(g_1 + .. + g_t) h_0."""
    rng = np.random.default_rng(0)
    x, g, h0 = rng.normal(size=(2, 9, 3)), -rng.random((2, 9, 3)), rng.normal(size=(2, 3))
    G = np.cumsum(g, axis=1)
    h, final, _, _ = ops.scan(x, g, h0)
    for t in range(9):
        w = np.exp(G[:, t:t + 1] - G[:, :t + 1])
        ref = (w * x[:, :t + 1]).sum(1) + np.exp(G[:, t]) * h0
        assert np.allclose(h[:, t], ref, rtol=1e-13, atol=1e-13)
    assert np.array_equal(final, h[:, -1])


def test_scan_packed_is_sequence_by_sequence():
    rng = np.random.default_rng(1)
    cu = [0, 0, 3, 4, 4, 9]
    x, g, h0 = rng.normal(size=(1, 9, 2)), -rng.random((1, 9, 2)), rng.normal(size=(5, 2))
    h, final, _, _ = ops.scan(x, g, h0, cu)
    for n in range(5):
        a, b = cu[n], cu[n + 1]
        if a == b:
            assert np.array_equal(final[n], h0[n])
            continue
        hn, fn, _, _ = ops.scan(x[:, a:b], g[:, a:b], h0[n:n + 1])
        assert np.array_equal(h[:, a:b], hn) and np.array_equal(final[n:n + 1], fn)


def _differences(f, arrays, eps=1e-6):
    """d f / d array by central differences, f a scalar function of the arrays."""
    out = []
    for i, a in enumerate(arrays):
        if a is None:
            out.append(None)
            continue
        d = np.zeros(a.shape)
        for ix in np.ndindex(a.shape):
            keep = a[ix]
            a[ix] = keep + eps
            up = f(*arrays)
            a[ix] = keep - eps
            down = f(*arrays)
            a[ix] = keep
            d[ix] = (up - down) / (2 * eps)
        out.append(d)
    return out


@pytest.mark.parametrize("cu", [None, [0, 0, 3, 4, 7]])
def test_scan_gradients_are_differences(cu):
    rng = np.random.default_rng(2)
    B, T, D, N = (2, 7, 2, 2) if cu is None else (1, 7, 2, 4)
    x, g = rng.normal(size=(B, T, D)), -rng.random((B, T, D))
    h0, wo, wf = rng.normal(size=(N, D)), rng.normal(size=(B, T, D)), rng.normal(size=(N, D))

    def loss(x, g, h0):
        h, final, _, _ = ops.scan(x, g, h0, cu)
        return (h * wo).sum() + (final * wf).sum()

    h = ops.scan(x, g, h0, cu)[0]
    got, _ = ops.scan_bwd(g, h, wo, h0, cu, wf)
    for a, b in zip(got, _differences(loss, [x, g, h0])):
        assert np.allclose(a, b, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("parts", ["w", "z", "r", "wz", "wzr", "rsn", "wrn", "wzrsn"])
def test_norm_gradients_are_differences(parts, kind):
    rng = np.random.default_rng(3)
    shape, d = (2, 3, 5), 5
    row = lambda on: rng.normal(size=shape) if on else None
    vec = lambda on: 1 + 0.3 * rng.normal(size=d) if on else None
    y, w, z, r = row(True), vec("w" in parts), row("z" in parts), row("r" in parts)
    s, nw = vec("s" in parts), vec("n" in parts)
    dout = row(r is None or nw is not None)
    drout = row(r is not None)

    def loss(y, w, z, r, s, nw):
        (out, rp), _ = ops.norm(y, w, z, kind, r, s, nw, 1e-3)
        return (0 if out is None else (out * dout).sum()) + (0 if rp is None else (rp * drout).sum())

    got, _ = ops.norm_bwd(y, dout, w, z, kind, r, s, nw, drout, 1e-3)
    want = dict(zip(("y", "weight", "gate", "residual", "scale", "next"),
                    _differences(loss, [y, w, z, r, s, nw])))
    assert set(got) == {k for k, v in want.items() if v is not None}
    for name, a in got.items():
        assert np.allclose(a, want[name], rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("rule", ["delta", "gdn", "kda", "gdp"])
def test_delta_step_is_the_token_recurrence(rule):
    """Against the C oracle of the forward pass, through a permuted cache."""
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen)
    N, T, H, dk, dv, nh = 3, 5, 2, 64, 128, 2 if rule == "gdp" else 1
    q, k, v = (torch.nn.functional.normalize(r(N, t, H, d), dim=-1) for t, d in
               ((T, dk), (T * nh, dk), (T * nh, dv)))
    beta, s0 = torch.sigmoid(r(N, T * nh, H)), r(N, H, dk, dv)
    g = {"delta": None, "gdn": -r(N, T, H).abs(), "gdp": -r(N, T, H).abs(),
         "kda": -r(N, T, H, dk).abs()}[rule]
    slots = [4, 0, 2]
    state = np.zeros((5, H, dk, dv))
    state[slots] = s0.numpy()
    (out, new), _ = ops.delta_step(*(t.double().numpy() for t in (q, k, v, beta)), state,
                                   None if g is None else g.double().numpy(), nh, slots)
    ref_o, ref_s = oracle.token_recurrence(q, k, v, beta, s0, g=g, n_sub=nh)
    assert np.allclose(out, ref_o.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(new[slots], ref_s.numpy(), rtol=1e-12, atol=1e-12)
    assert not new[[1, 3]].any()


def test_delta_step_padding_and_repeated_slots():
    rng = np.random.default_rng(5)
    q, k, v = (rng.normal(size=(5, 1, 1, d)) for d in (64, 64, 64))
    beta, state = rng.random((5, 1, 1)), rng.normal(size=(3, 1, 64, 64))
    (out, new), _ = ops.delta_step(q, k, v, beta, state, slots=[1, -1, 1, 7, 0])
    assert np.array_equal(new[2], state[2])
    assert not out[[1, 2, 3]].any() and out[[0, 4]].any()
    (_, alone), _ = ops.delta_step(q[:1], k[:1], v[:1], beta[:1], state, slots=[1])
    assert np.array_equal(new[1], alone[1])
