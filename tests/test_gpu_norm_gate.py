"""The gate's gradient of deltanet_norm_bwd where the sigmoid saturates.

Tolerance, relative: with U = 2^-24 the exponential carries (4 + 2.4 |z|) U and enters up to three
times (itself and the two s = 1 / (1 + e)), each s another 5 U (its sum, its quotient), the four
products 4 U: (26 + 7.2 |z|) U, and half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("d", [1, 64, 333, 2048, 5000])
def test_the_sigmoids_derivative_keeps_its_figures(d, dtype):
    rows = max(2, 4096 // d)
    gen = torch.Generator().manual_seed(d)
    z = torch.linspace(-80, 80, rows * d, dtype=torch.float64).view(rows, d).to(DEV, dtype)
    y, dout = ((1 + torch.rand((rows, d), generator=gen)).to(DEV, dtype) for _ in range(2))
    gr = dn.deltanet_norm_bwd(y, dout, None, z, activation="sigmoid")
    f64 = lambda t: t.double().cpu().numpy()
    zz = f64(z)
    s, rest = 1 / (1 + np.exp(-zz)), 1 / (1 + np.exp(zz))
    for got, want in ((gr.d_gate, f64(dout) * f64(y) * s * rest), (gr.d_y, f64(dout) * s)):
        tol = ((26 + 7.2 * np.abs(zz)) * 2.0 ** -24 + HALF[dtype]) * np.abs(want)
        bad = ~(np.abs(f64(got) - want) <= tol)
        assert not bad.any(), (zz[bad][:4], f64(got)[bad][:4], want[bad][:4])


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gates_at_the_ends(activation):
    """Infinite gates and NaN: what the formula gives, 0 or 1 and its derivative 0; silu of -inf is
    -inf times 0."""
    z = torch.tensor([[float("inf"), float("-inf"), float("nan"), 200.0, -200.0, 88.5, -88.5, 0.0]], device=DEV)
    y = torch.full_like(z, 2.0)
    gr = dn.deltanet_norm_bwd(y, torch.ones_like(y), None, z, activation=activation)
    dz, dy = gr.d_gate[0].tolist(), gr.d_y[0].tolist()
    assert np.isnan(dz[2]) and np.isnan(dy[2])
    if activation == "sigmoid":
        assert dz[:2] == [0, 0] and dy[:2] == [1, 0] and dy[3:5] == [1, 0] and dz[7] == 0.5
        assert max(map(abs, dz[3:7])) < 1e-37 and dy[7] == 0.5
    else:
        assert np.isnan(dy[1]) and dy[3:5] == [200, 0] and dz[3] == 2 and dz[7] == 1 and dy[7] == 0
