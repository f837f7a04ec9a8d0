"""The error word of a stream, which deltanet_get_error reads, and the workspace beside it: reports
reach the caller whatever other streams do meanwhile, and captured calls leave both sound."""
import contextlib
import ctypes

import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn
from deltanet_chunkwise_delta_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


@contextlib.contextmanager
def new_stream():
    """A non-blocking stream that never had a call (torch's own come from a pool)."""
    torch.cuda.current_stream()                        # there is a context
    driver, handle = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
    assert driver.cuStreamCreate(ctypes.byref(handle), 1) == 0
    s = torch.cuda.ExternalStream(handle.value)
    yield s
    s.synchronize()                                    # kept: its handle must not come again


def rnd(*shape, dtype=BF, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def bad_slot():
    x, g, cache = rnd(2, 1, 64), -rnd(2, 1, 64, dtype=F).abs(), rnd(2, 64, dtype=F)
    slots, out = torch.tensor([1, 7], dtype=torch.int32, device=DEV), torch.empty_like(x)
    return lambda: dn.deltanet_scan_step(x, g, cache, slots, out=out)


def bad_boundary():
    x, g, cu = rnd(1, 40, 64), -rnd(1, 40, 64, dtype=F).abs(), torch.tensor([0, 30, 39], dtype=torch.int32, device=DEV)
    out, fin = torch.empty_like(x), torch.empty((2, 64), device=DEV)
    return lambda: dn.deltanet_scan_fwd(x, g, None, cu, out, fin)


def busy_default_stream():
    """About 0.3 s of work on the default stream, behind which a memset there would wait."""
    torch.cuda._sleep(600_000_000)


@pytest.mark.parametrize("kind,error", [(bad_slot, L.DN_ERR_SLOTS), (bad_boundary, L.DN_ERR_SEQLENS)])
def test_reports_while_the_default_stream_is_busy(kind, error):
    """The stream's first call, which makes its word, and a call after a report was read."""
    call = kind()
    call()                                             # the kernel is loaded, which waits for the GPU
    assert dn.get_error() == error
    with new_stream() as s:
        for _ in range(2):
            torch.cuda.synchronize()
            busy_default_stream()
            with torch.cuda.stream(s):
                call()
                assert dn.get_error(s) == error        # read and cleared ..
                call()
                torch.cuda.synchronize()               # .. once, whatever else was under way
                assert dn.get_error(s) == error
                assert dn.get_error(s) == 0


def test_a_workspace_does_not_grow_inside_a_capture():
    """A stream that had a token step (its error word exists, a workspace does not): the chunkwise
    call captured on it is refused and the capture goes on; after a call of its size it is taken,
    and eager calls, replays and larger calls follow in any order."""
    q, k, v = (rnd(1, 200, 2, 128, seed=s) * 0.1 for s in (1, 2, 3))
    beta = rnd(1, 200, 2, dtype=F, seed=4).sigmoid()
    want, wfin = dn.deltanet_fwd(q, k, v, beta)
    torch.cuda.synchronize()
    with new_stream() as s:
        with torch.cuda.stream(s):
            bad_slot()()
            assert dn.get_error(s) == L.DN_ERR_SLOTS
        t = torch.zeros(1, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(dn.DeltaNetError) as e:
                dn.deltanet_fwd(q, k, v, beta)
            t += 1
        assert e.value.status == L.DN_ERR_WORKSPACE
        graph.replay()
        torch.cuda.synchronize()
        assert t.item() == 1
        with torch.cuda.stream(s):
            out, fin = dn.deltanet_fwd(q, k, v, beta)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(fin, wfin)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, fin = dn.deltanet_fwd(q, k, v, beta)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(fin, wfin)
        assert dn.get_error(s) == 0


def test_captured_steps_outlive_the_workspaces():
    """deltanet_release_workspace leaves what a captured step reports to."""
    with new_stream() as s:
        call = bad_slot()
        with torch.cuda.stream(s):
            call()
            assert dn.get_error(s) == L.DN_ERR_SLOTS
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        dn.release_workspace()
        torch.cuda.empty_cache()
        with torch.cuda.stream(s):
            graph.replay()
            assert dn.get_error(s) == L.DN_ERR_SLOTS
            assert dn.get_error(s) == 0


@pytest.mark.parametrize("kind,error", [(bad_slot, L.DN_ERR_SLOTS), (bad_boundary, L.DN_ERR_SEQLENS)])
def test_the_first_call_on_a_stream_may_be_captured(kind, error):
    """As decoding is captured: nothing ran on the capture's stream before.  Every replay reports,
    on any stream, and a report stays until it is read."""
    call = kind()
    call()
    assert dn.get_error() == error
    with new_stream() as s:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        assert dn.get_error(s) == 0                    # captured, not run
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert dn.get_error(s) == error
            assert dn.get_error(s) == 0
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert dn.get_error(s) == error and dn.get_error() == 0


def test_steps_captured_on_torchs_own_stream():
    """torch.cuda.graph() without a stream, the usual way, and two graphs from it."""
    x, g = rnd(3, 1, 64), -rnd(3, 1, 64, dtype=F).abs()
    slots = torch.tensor([2, 0, 4], dtype=torch.int32, device=DEV)
    caches = [rnd(5, 64, dtype=F, seed=s) for s in (1, 2)]
    want = [c.clone() for c in caches]
    outs = [[dn.deltanet_scan_step(x, g, c, slots) for _ in range(3)] for c in want]
    graphs, got = [], []
    for c in caches:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(dn.deltanet_scan_step(x, g, c, slots))
    for t in range(3):
        for i in (0, 1):
            graphs[i].replay()
            assert torch.equal(got[i], outs[i][t])
    assert all(torch.equal(a, b) for a, b in zip(caches, want)) and dn.get_error() == 0
