"""Host-side checks of deltanet_step, deltanet_scan_* and deltanet_norm_*: bad arguments are
refused before a GPU is touched (these calls never reach the device)."""
import ctypes

import pytest
import torch

from deltanet_chunkwise_delta_b200 import _lib as L
from deltanet_chunkwise_delta_b200 import build as B
import deltanet_chunkwise_delta_b200 as dn

ARG, UNS, ALIAS = L.DN_ERR_INVALID_ARG, L.DN_ERR_UNSUPPORTED, L.DN_ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def desc(shape, dtype=L.DN_BF16, at=1, strides=None, off=0):
    """A descriptor at address `at` * 256 MB + off."""
    d = L.DnTensor()
    d.data, d.dtype, d.ndim = at * 2**28 + off, dtype, len(shape)
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    for i, (s, st) in enumerate(zip(shape, strides)):
        d.shape[i], d.stride[i] = s, st
    return d


def ref(x):
    return None if x is None else ctypes.addressof(x)


class Step:
    def __init__(self, N=3, T=2, H=2, dk=128, dv=64, nh=1, M=5, dtype=L.DN_BF16):
        self.a = dict(q=desc([N, T, H, dk], dtype, 1), k=desc([N, T * nh, H, dk], dtype, 2),
                      v=desc([N, T * nh, H, dv], dtype, 3), beta=desc([N, T * nh, H], L.DN_F32, 4),
                      g=None, n_h=nh, state=desc([M, H, dk, dv], L.DN_F32, 6),
                      slot_idx=desc([N], L.DN_I32, 7), out=desc([N, T, H, dv], dtype, 8))

    def __call__(self, lib, **kw):
        a = {**self.a, **kw}
        return lib.deltanet_step(*[x if n == "n_h" else ref(x) for n, x in a.items()], None)


# Refusals only: a call that is accepted would launch on made-up addresses where there is a device.
def test_step_refusals(lib):
    s = Step()
    for name in ("q", "k", "v", "beta", "state", "out"):
        assert s(lib, **{name: None}) == ARG, name
    assert s(lib, n_h=0) == ARG and s(lib, n_h=2) == ARG          # k has one row per token
    assert s(lib, k=desc([3, 2, 2, 64], at=2)) == ARG
    assert s(lib, out=desc([3, 2, 2, 64], L.DN_F32, 8)) == ARG
    assert s(lib, beta=desc([3, 2, 2], L.DN_BF16, 4)) == ARG
    assert s(lib, g=desc([3, 2], L.DN_F32, 5)) == ARG
    assert s(lib, g=desc([3, 2, 2], L.DN_BF16, 5)) == ARG
    assert s(lib, g=desc([3, 2, 2, 64], L.DN_F32, 5)) == ARG      # per key channel: d_k values
    assert s(lib, g=desc([3, 2, 2, 128], L.DN_F32, 5, off=4)) == ARG
    assert s(lib, q=desc([3, 2, 2, 128], off=2)) == ARG           # 16-byte rows
    assert s(lib, state=desc([5, 2, 128, 64], L.DN_BF16, 6)) == ARG
    assert s(lib, state=desc([5, 2, 64, 128], L.DN_F32, 6)) == ARG
    assert s(lib, slot_idx=desc([4], L.DN_I32, 7)) == ARG
    assert s(lib, slot_idx=desc([3], L.DN_F32, 7)) == ARG
    assert s(lib, slot_idx=None) == ARG                           # 3 requests, 5 rows
    # state rows on top of each other
    assert s(lib, state=desc([5, 2, 128, 64], L.DN_F32, 6, strides=[0, 8192, 64, 1])) == ARG
    assert s(lib, state=desc([5, 2, 128, 64], L.DN_F32, 6, strides=[8192, 8192, 64, 1])) == ARG
    assert s(lib, out=desc([3, 2, 2, 64], at=6, off=4096)) == ALIAS
    assert s(lib, out=desc([3, 2, 2, 64], at=1)) == ALIAS
    assert s(lib, slot_idx=desc([3], L.DN_I32, 6, off=64)) == ALIAS
    assert Step(dk=96)(lib) == UNS and Step(dv=256)(lib) == UNS
    assert Step(N=2**16, T=2**15, H=1, nh=1, M=2**16)(lib) == ARG            # N T n_h reaches 2^31
    assert Step(N=2**20, T=0, H=2**12, M=2**20)(lib, slot_idx=None) == ARG   # more CTAs than a grid has


def scan_args(B=2, T=9, D=10, N=None, x=L.DN_BF16, g=L.DN_F32):
    N = B if N is None else N
    return dict(x=desc([B, T, D], x, 1), g=desc([B, T, D], g, 2), s0=desc([N, D], L.DN_F32, 3), cu=None,
                out=desc([B, T, D], x, 4), fin=desc([N, D], L.DN_F32, 5))


def test_scan_fwd_refusals(lib):
    a = scan_args()
    f = lambda **kw: lib.deltanet_scan_fwd(*[ref(x) for x in {**a, **kw}.values()], None)
    for name in ("x", "g", "out"):
        assert f(**{name: None}) == ARG, name
    assert f(g=desc([2, 9, 11], L.DN_F32, 2)) == ARG
    assert f(x=desc([2, 9, 10], L.DN_F32), out=desc([2, 9, 10], L.DN_F32, 4),
             g=desc([2, 9, 10], L.DN_BF16, 2)) == ARG             # bf16 gates need bf16 x
    assert f(out=desc([2, 9, 10], L.DN_F32, 4)) == ARG
    assert f(s0=desc([2, 10], L.DN_BF16, 3)) == ARG and f(fin=desc([3, 10], L.DN_F32, 5)) == ARG
    assert f(x=desc([2, 9, 10], strides=[90, 10, 2])) == ARG
    assert f(x=desc([2, 9, 10], strides=[90, -10, 1])) == ARG
    assert f(x=desc([2, 9, 10], off=1)) == ARG and f(g=desc([2, 9, 10], L.DN_F32, 2, off=2)) == ARG
    assert f(x=desc([2, 9], L.DN_BF16)) == ARG
    assert f(cu=desc([3], L.DN_I32, 6)) == ARG                    # packed input has one row
    assert f(out=desc([2, 9, 10], at=4, strides=[0, 10, 1])) == ARG
    assert f(out=desc([2, 9, 10], at=4, strides=[90, 5, 1])) == ARG
    assert f(out=desc([2, 9, 10], at=1)) == ALIAS                 # in place: refused
    assert f(out=desc([2, 9, 10], at=1, off=16)) == ALIAS
    assert f(fin=desc([2, 10], L.DN_F32, 3)) == ALIAS
    # interleaved rows in one buffer that do touch: 10 values in a pitch of 15
    assert f(x=desc([2, 9, 10], strides=[135, 15, 1]),
             out=desc([2, 9, 10], at=1, off=10, strides=[135, 15, 1])) == ALIAS
    p = scan_args(B=1, N=2)
    g = lambda **kw: lib.deltanet_scan_fwd(*[ref(x) for x in {**p, **kw}.values()], None)
    assert g(cu=desc([3], L.DN_F32, 6)) == ARG and g(cu=desc([4], L.DN_I32, 6)) == ARG
    assert g(cu=desc([0], L.DN_I32, 6)) == ARG
    assert g(cu=desc([3], L.DN_I32, 5)) == ALIAS


def test_scan_bwd_and_step_refusals(lib):
    a = dict(g=desc([2, 9, 10], L.DN_F32, 1), out=desc([2, 9, 10], at=2), s0=None, cu=None,
             d_out=desc([2, 9, 10], at=3), d_fin=None, d_x=desc([2, 9, 10], at=4),
             d_g=desc([2, 9, 10], L.DN_F32, 5), d_s0=None)
    f = lambda **kw: lib.deltanet_scan_bwd(*[ref(x) for x in {**a, **kw}.values()], None)
    for name in ("g", "out", "d_out", "d_x", "d_g"):
        assert f(**{name: None}) == ARG, name
    assert f(d_out=desc([2, 9, 10], L.DN_F32, 3)) == ARG
    assert f(d_g=desc([2, 9, 10], L.DN_BF16, 5)) == ARG
    assert f(d_fin=desc([2, 11], L.DN_F32, 6)) == ARG
    assert f(d_x=desc([2, 9, 10], at=3)) == ALIAS and f(d_g=desc([2, 9, 10], L.DN_F32, 1)) == ALIAS
    assert f(d_fin=desc([2, 10], L.DN_F32, 6), d_s0=desc([2, 10], L.DN_F32, 6)) == ALIAS
    b = dict(x=desc([3, 1, 10], at=1), g=desc([3, 1, 10], L.DN_F32, 2), state=desc([4, 10], L.DN_F32, 3),
             slot_idx=desc([3], L.DN_I32, 4), out=desc([3, 1, 10], at=5))
    s = lambda **kw: lib.deltanet_scan_step(*[ref(x) for x in {**b, **kw}.values()], None)
    for name in ("x", "g", "state", "out"):
        assert s(**{name: None}) == ARG, name
    assert s(slot_idx=None) == ARG and s(slot_idx=desc([2], L.DN_I32, 4)) == ARG
    assert s(state=desc([4, 11], L.DN_F32, 3)) == ARG
    assert s(state=desc([4, 10], L.DN_F32, 3, strides=[0, 1])) == ARG
    assert s(state=desc([4, 10], L.DN_F32, 2)) == ALIAS and s(out=desc([3, 1, 10], at=3)) == ALIAS


def norm_args(shape=(3, 4, 24), y=L.DN_BF16, r=L.DN_BF16):
    d = [shape[-1]]
    return dict(y=desc(shape, y, 1), w=desc(d, L.DN_F32, 2), gate=desc(shape, y, 3), act=0,
                res=desc(shape, r, 4), sc=desc(d, L.DN_BF16, 5), nw=desc(d, L.DN_F32, 6), eps=1e-6,
                out=desc(shape, y, 7), rout=desc(shape, r, 8))


def call_args(a):
    return [x if n in ("act", "eps") else ref(x) for n, x in a.items()]


def test_norm_fwd_refusals(lib):
    a, sh = norm_args(), (3, 4, 24)
    f = lambda **kw: lib.deltanet_norm_fwd(*call_args({**a, **kw}), None)
    assert f(y=None) == ARG and f(out=None) == ARG and f(rout=None) == ARG
    assert f(res=None) == ARG                                     # scale, next_weight, rout need it
    assert f(res=None, sc=None, nw=None) == ARG                   # rout is still given
    assert f(nw=None) == ARG                                      # out is still given
    assert f(w=None, gate=None, res=None, sc=None, nw=None, rout=None) == ARG
    assert f(act=2) == ARG and f(act=-1) == ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == ARG
    assert f(gate=desc(sh, L.DN_F32, 3)) == ARG                   # gate has y's dtype
    b = norm_args(y=L.DN_F32, r=L.DN_F32)
    assert lib.deltanet_norm_fwd(*call_args({**b, "res": desc(sh, L.DN_BF16, 4)}), None) == ARG
    assert f(rout=desc(sh, L.DN_F32, 8)) == ARG and f(out=desc(sh, L.DN_F32, 7)) == ARG
    assert f(w=desc([23], L.DN_F32, 2)) == ARG and f(sc=desc([24], L.DN_I32, 5)) == ARG
    assert f(nw=desc([24], L.DN_F32, 6, strides=[2])) == ARG
    assert f(y=desc((24,), at=1)) == ARG
    assert f(out=desc(sh, at=7, strides=[0, 24, 1])) == ARG
    assert f(out=desc(sh, at=1)) == ALIAS and f(rout=desc(sh, at=4)) == ALIAS
    assert f(out=desc(sh, at=8)) == ALIAS
    big = norm_args((1, 16385))
    assert lib.deltanet_norm_fwd(*call_args(big), None) == UNS


def test_norm_bwd_refusals(lib):
    a, sh, d = norm_args(), (3, 4, 24), [24]
    for n in ("out", "rout"):
        a.pop(n)
    a.update(d_out=desc(sh, at=9), d_rout=desc(sh, at=10), d_y=desc(sh, at=11), d_w=desc(d, L.DN_F32, 12),
             d_gate=desc(sh, at=13), d_res=desc(sh, at=14), d_sc=desc(d, L.DN_F32, 15),
             d_nw=desc(d, L.DN_F32, 16))
    n = lib.deltanet_norm_workspace(12, 24)
    a["work"] = desc([n], L.DN_F32, 17)
    f = lambda **kw: lib.deltanet_norm_bwd(*call_args({**a, **kw}), None)
    for name in ("y", "d_out", "d_y", "d_w", "d_gate", "d_res", "d_sc", "d_nw", "work"):
        assert f(**{name: None}) == ARG, name
    assert f(w=None) == ARG                                       # its gradient is still asked for
    assert f(nw=None, d_nw=None, d_out=None, d_rout=None) == ARG  # nothing to differentiate
    assert f(d_w=desc(d, L.DN_BF16, 12)) == ARG
    assert f(d_res=desc(sh, L.DN_F32, 14)) == ARG
    assert f(work=desc([n], L.DN_F32, 17, off=4)) == ARG
    assert f(work=desc([n - 1], L.DN_F32, 17)) == L.DN_ERR_WORKSPACE
    assert f(work=desc([n], L.DN_F32, 11)) == ALIAS
    assert f(d_y=desc(sh, at=1)) == ALIAS and f(d_w=desc(d, L.DN_F32, 15)) == ALIAS
    assert lib.deltanet_norm_workspace(0, 24) == 0 and n >= 3 * 24


def test_bindings_refuse_cpu_tensors_and_unknown_activations():
    x = torch.zeros(1, 4, 64)
    s = torch.zeros(1, 64)
    q, b, st = torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1), torch.zeros(1, 1, 64, 64)
    for f in (lambda: dn.deltanet_scan_fwd(x, x), lambda: dn.deltanet_scan_bwd(x, x, x),
              lambda: dn.deltanet_scan_step(x, x, s), lambda: dn.deltanet_step(q, q, q, b, st),
              lambda: dn.deltanet_norm_fwd(x, torch.ones(64)),
              lambda: dn.deltanet_norm_bwd(x, x, torch.ones(64)),
              lambda: dn.deltanet_norm_fwd(x, activation="relu")):
        with pytest.raises(ValueError):
            f()


def test_descriptor_bytes_are_the_struct():
    """The packed descriptors hold what the ctypes structure holds."""
    t = torch.zeros(3, 4, 10)[:, :, 2:7]
    u = torch.zeros(6, dtype=torch.int32)
    addr = L._descriptors(t, None, u)
    assert addr[1] is None
    for a, x in ((addr[0], t), (addr[2], u)):
        d, e = L.DnTensor.from_address(a), L.describe(x)
        assert (d.data, d.dtype, d.ndim) == (e.data, e.dtype, e.ndim)
        assert list(d.shape) == list(e.shape) and list(d.stride) == list(e.stride)
    with pytest.raises(TypeError):
        L._descriptors(torch.zeros(2, dtype=torch.float16))


def test_short_calls_leave_cpu_tensors_to_the_general_way(lib):
    c = L._short()
    t = torch.zeros(2, 3, 4)
    assert c.scan_step(t, t, t[0], None, None) is None
    assert c.norm_fwd(t, None, None, None, None, None, 0, 1e-6, None, None) is None
    assert c.scan_fwd(None, t, None, None, None, None, True) is None
    with pytest.raises(TypeError):
        c.step(t)


def test_status_string_of_slots():
    assert L.status_string(L.DN_ERR_SLOTS).startswith("DN_ERR_SLOTS")
