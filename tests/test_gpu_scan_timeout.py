"""The gated linear recurrence when a wait inside a cluster gives up, with no fault: the library's
test hook (deltanet_test_set_wait) lets the first CTA of every cluster send the others nothing at
one tile, so that all their waits for it run out after a short limit.  They stop, what they had
under way lands, the call reports DN_ERR_TIMEOUT, and a normal call follows."""
import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn
from deltanet_chunkwise_delta_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
LIMIT_NS = 1_000_000  # 1 ms


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()
    yield
    dn.test_set_wait()


def inputs(T, D, x, g, N=1):
    gen = torch.Generator().manual_seed(T + D)
    r = lambda *s: torch.randn(s, generator=gen)
    return (r(1, T, D).to(DEV, x), (-r(1, T, D).abs() * 0.3).to(DEV, g), r(N, D).to(DEV), r(1, T, D).to(DEV, x))


def stalled(tile, call):
    dn.test_set_wait(LIMIT_NS, tile + 1)
    try:
        got = call()
        assert dn.get_error() == L.DN_ERR_TIMEOUT
    finally:
        dn.test_set_wait()
    assert dn.get_error() == 0                         # read once, then cleared
    return got


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@pytest.mark.parametrize("x,g", [(BF, F), (BF, BF), (F, F)])
@pytest.mark.parametrize("tile", [0, 1, 4])
@pytest.mark.parametrize("T,D", [(6000, 64), (900, 640), (6000, 33)])
def test_dense(T, D, x, g, tile):
    """Tokens ahead of the tile are right, the others (backward: those before it) NaN; clusters of
    eight and of two, one and several to a call, odd rows."""
    xs, gs, s0, dh = inputs(T, D, x, g)
    fwd = lambda: dn.deltanet_scan_fwd(xs, gs, s0)
    want = fwd()
    bwd = lambda: dn.deltanet_scan_bwd(gs, want[0], dh, s0)
    wantb = bwd()
    assert dn.get_error() == 0
    tiles = 0
    for call, ref, back in ((fwd, want, False), (bwd, wantb, True)):
        dn.test_set_wait(LIMIT_NS, tile + 1)
        try:
            got = call()
            status = dn.get_error()
        finally:
            dn.test_set_wait()
        if status == 0:                                # the row has no such tile
            assert tile > 0 and same(got, ref)
            continue
        tiles += 1
        assert status == L.DN_ERR_TIMEOUT and dn.get_error() == 0
        out, whole = (got[0].flip(1), ref[0].flip(1)) if back else (got[0], ref[0])
        lost = torch.isnan(out[0])
        first = int(lost[:, 0].int().argmax())
        assert lost[first:].all() and not lost[:first].any()
        assert torch.equal(out[0, :first], whole[0, :first])
        assert (first == 0) == (tile == 0) and torch.isnan(got[-1]).all()
        assert same(call(), ref)
    assert tiles == 2 or (tile == 4 and T == 900)
    assert dn.get_error() == 0


@pytest.mark.parametrize("x,g", [(BF, F), (F, F)])
@pytest.mark.parametrize("tile", [0, 2])
def test_packed(x, g, tile):
    """Every token is right or NaN, and sequences without a token of the tile or after it right."""
    cu = [0, 37, 37, 400, 1500, 2600, 2601, 4000]
    xs, gs, s0, dh = inputs(4000, 64, x, g, len(cu) - 1)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    fwd = lambda: dn.deltanet_scan_fwd(xs, gs, s0, c)
    want = fwd()
    bwd = lambda: dn.deltanet_scan_bwd(gs, want[0], dh, s0, c, s0)
    wantb = bwd()
    for call, ref in ((fwd, want), (bwd, wantb)):
        got = stalled(tile, call)
        assert torch.isnan(got[0]).any()
        for a, b in zip(got, ref):
            lost = torch.isnan(a)
            assert torch.equal(a[~lost], b[~lost])
        assert same(call(), ref)
    assert dn.get_error() == 0


def test_a_short_limit_alone_changes_nothing():
    xs, gs, s0, dh = inputs(6000, 640, BF, F)
    want = dn.deltanet_scan_fwd(xs, gs, s0)
    dn.test_set_wait(LIMIT_NS, 0)
    try:
        got = dn.deltanet_scan_fwd(xs, gs, s0)
        back = dn.deltanet_scan_bwd(gs, want[0], dh, s0)
        assert dn.get_error() == 0
    finally:
        dn.test_set_wait()
    assert same(got, want) and same(back, dn.deltanet_scan_bwd(gs, want[0], dh, s0))
