"""The two ways from Python into the operators around the mixers: the short one (the current
stream) and the general one (a stream is named) make the same call."""
import sys
import threading

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


def rnd(*shape, dtype=BF, seed=0, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(DEV, dtype)


def slots(*ids):
    return torch.tensor(ids, dtype=torch.int32, device=DEV)


def calls():
    """(name, f(stream, outputs...)) with f's results, and what buffers the outputs may be."""
    q, k, v = rnd(3, 2, 4, 64, seed=1), rnd(3, 2, 4, 64, seed=2, scale=0.1), rnd(3, 2, 4, 128, seed=3)
    beta, g = rnd(3, 2, 4, dtype=F, seed=4).sigmoid(), -rnd(3, 2, 4, dtype=F, seed=5).abs()
    cache = rnd(6, 4, 64, 128, dtype=F, seed=6)
    x, gx, h0 = rnd(1, 700, 192, seed=7), -rnd(1, 700, 192, dtype=F, seed=8).abs(), rnd(3, 192, dtype=F, seed=9)
    cu = torch.tensor([0, 100, 100, 700], dtype=torch.int32, device=DEV)
    xs, gs, hs = rnd(4, 3, 96, seed=10), -rnd(4, 3, 96, seed=11).abs(), rnd(5, 96, dtype=F, seed=12)
    y, z, r = rnd(5, 7, 256, seed=13), rnd(5, 7, 256, seed=14), rnd(5, 7, 256, dtype=F, seed=15)
    w, sc, nw = (rnd(256, dtype=F, seed=s) for s in (16, 17, 18))

    def step(**kw):
        c = cache.clone()
        return dn.deltanet_step(q, k, v, beta, c, g, slot_idx=slots(5, -1, 0), **kw), c

    def scan_step(**kw):
        c = hs.clone()
        return dn.deltanet_scan_step(xs, gs, c, slots(1, 4, -1, 0), **kw), c

    def scan_bwd(**kw):
        h, _ = dn.deltanet_scan_fwd(x, gx, h0, cu)
        return dn.deltanet_scan_bwd(gx, h, x, h0, cu, d_final_state=h0, **kw)

    e = torch.empty_like
    return [("step", step, dict(out=e(v))), ("scan_step", scan_step, dict(out=e(xs))),
            ("scan_fwd", lambda **kw: dn.deltanet_scan_fwd(x, gx, h0, cu, **kw), dict(out=e(x), final_state=e(h0))),
            ("scan_fwd_dense", lambda **kw: dn.deltanet_scan_fwd(x, gx, output_final_state=False, **kw), dict(out=e(x))),
            ("scan_bwd", scan_bwd, dict(d_x=e(x), d_g=e(gx), d_initial_state=e(h0))),
            ("norm", lambda **kw: dn.deltanet_norm_fwd(y, w, **kw), dict(out=e(y))),
            ("norm_fwd", lambda **kw: dn.deltanet_norm_fwd(y, w, z, r, sc, nw, activation="sigmoid", eps=1e-5, **kw),
             dict(out=e(y), residual_out=e(r))),
            ("norm_residual", lambda **kw: dn.deltanet_norm_fwd(y, None, z, r, **kw), dict(residual_out=e(r))),
            ("norm_bwd", lambda **kw: dn.deltanet_norm_bwd(y, z, w, z, r, sc, nw, r, activation="sigmoid", eps=1e-5, **kw),
             dict(d_y=e(y), d_gate=e(z), d_residual=e(r))),
            ("norm_bwd_head", lambda **kw: dn.deltanet_norm_bwd(y, z, w, z, **kw), dict(d_y=e(y), d_gate=e(z)))]


def flat(r):
    return [t for x in r for t in (flat(x) if isinstance(x, tuple) else [x])] if isinstance(r, tuple) else [r]


def same(a, b):
    a, b = flat(a), flat(b)
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


@pytest.mark.parametrize("i", range(10))
def test_both_ways_are_one_call(i):
    name, f, outs = calls()[i]
    short = f()
    here = torch.cuda.current_stream()
    same(short, f(stream=here))
    a, b = ({n: torch.full_like(t, 7) for n, t in outs.items()} for _ in range(2))
    ra, rb = f(**a), f(stream=here, **b)
    same(ra, short)
    same(rb, short)
    for n in outs:                                     # the caller's buffers are what comes back
        assert any(t is a[n] for t in flat(ra)) and any(t is b[n] for t in flat(rb))
    assert type(ra) is type(rb) is type(short)


def test_refusals_are_the_same_both_ways():
    q, k, v = rnd(3, 2, 4, 64), rnd(3, 2, 4, 64), rnd(3, 2, 4, 64)
    beta, cache, h = rnd(3, 2, 4, dtype=F), rnd(3, 4, 64, 64, dtype=F), rnd(2, 5, 8)
    y, w = rnd(4, 64), rnd(64, dtype=F)
    bad = [(lambda **kw: dn.deltanet_step(q, k[:, :1], v, beta, cache, **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_step(q, k, v, beta, cache, out=v, **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_step(q, k, v, beta, cache.half(), **kw), TypeError),
           (lambda **kw: dn.deltanet_step(q, k, v, beta.cpu(), cache, **kw), ValueError),
           (lambda **kw: dn.deltanet_scan_fwd(h, h.float()[:, :4], **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_scan_fwd(h.double(), h.float(), **kw), TypeError),
           (lambda **kw: dn.deltanet_scan_bwd(h.float(), h, h, d_x=h, **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_scan_step(h, h, rnd(3, 8, dtype=F), **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_norm_fwd(y, w[:63], **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_norm_fwd(y, eps=-1.0, weight=w, **kw), dn.DeltaNetError),
           (lambda **kw: dn.deltanet_norm_fwd(y.view(2, 1, 1, 2, 64), w, **kw), ValueError),
           (lambda **kw: dn.deltanet_norm_bwd(y, None, w, **kw), dn.DeltaNetError)]
    for n, (f, err) in enumerate(bad):
        got = []
        for kw in ({}, dict(stream=torch.cuda.current_stream())):
            with pytest.raises(err) as e:
                f(**kw)
            got.append(getattr(e.value, "status", None))
        assert got[0] == got[1], n


def test_results_are_owned_once():
    y, w = rnd(64, 256), rnd(256, dtype=F)
    out, none = dn.deltanet_norm_fwd(y, w)
    buf = torch.empty_like(y)
    before = sys.getrefcount(buf)
    kept, _ = dn.deltanet_norm_fwd(y, w, out=buf)
    assert none is None and kept is buf and sys.getrefcount(buf) == before + 1
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    for _ in range(50):
        dn.deltanet_norm_bwd(y, y, w)
        with pytest.raises(dn.DeltaNetError):
            dn.deltanet_norm_fwd(y, w[:8])
    assert torch.cuda.memory_allocated() == base


def test_two_threads_on_streams_of_their_own():
    args = [(rnd(4, 1, 2, 64, seed=s), rnd(4, 1, 2, 64, seed=s + 1, scale=0.1), rnd(4, 1, 2, 64, seed=s + 2),
             rnd(4, 1, 2, dtype=F, seed=s + 3).sigmoid()) for s in (20, 30)]
    start = rnd(4, 2, 64, 64, dtype=F, seed=40)
    want = []
    for a in args:
        c = start.clone()
        for _ in range(40):
            o = dn.deltanet_step(*a, c)
        want.append((o, c))
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            c = start.clone()
            for _ in range(40):
                o = dn.deltanet_step(*args[i], c)
            torch.cuda.current_stream().synchronize()
            got[i] = (o, c)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    for w, g in zip(want, got):
        same(w, g)


def test_inputs_that_want_gradients():
    y, w = rnd(3, 64).requires_grad_(), rnd(64, dtype=F).requires_grad_()
    out, _ = dn.deltanet_norm_fwd(y, w)
    assert not out.requires_grad and L._call is not None
