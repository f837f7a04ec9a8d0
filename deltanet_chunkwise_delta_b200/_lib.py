"""ctypes binding of the C ABI in include/deltanet.h.

Argument marshalling only: torch tensors are described as ``dn_tensor``
structs (pointer, dtype, shape, strides in elements) and handed to the shared
library (the operators around the mixers by csrc/dn_call.cpp, where the call is
a plain one).  Every step of the computation runs in the library's CUDA kernels;
there is no other implementation to fall back to.  If the library is missing
or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import threading
import warnings
from typing import NamedTuple, Optional

import torch

from . import build as _build

DN_OK, DN_ERR_INVALID_ARG, DN_ERR_UNSUPPORTED, DN_ERR_ALIAS, DN_ERR_CUDA, \
    DN_ERR_WORKSPACE, DN_ERR_SEQLENS, DN_ERR_TIMEOUT, DN_ERR_SLOTS = range(9)
DN_F32, DN_BF16, DN_I32 = 0, 1, 2
DN_ACT_SILU, DN_ACT_SIGMOID = 0, 1

EXPORTED = ("deltanet_fwd", "deltanet_fwd_ex", "gated_deltanet_fwd", "gated_deltanet_fwd_ex",
            "gated_deltaproduct_fwd", "gated_deltaproduct_fwd_ex", "deltanet_fwd_states",
            "deltanet_status_string",
            "deltanet_get_error", "deltanet_release_workspace", "deltanet_last_schedule",
            "deltanet_fwd_noalloc", "deltanet_last_launches", "deltanet_set_kernel_events",
            "deltanet_test_set_wait", "kda_fwd", "kda_fwd_ex",
            "deltanet_step", "deltanet_scan_fwd", "deltanet_scan_bwd", "deltanet_scan_step",
            "deltanet_norm_fwd", "deltanet_norm_bwd", "deltanet_norm_workspace")


class DnTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class DeltaNetError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None):
    """Load the shared library (built in-tree by ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"DeltaNet CUDA library not found at {path}; run "
                "`python -m deltanet_chunkwise_delta_b200.build` (nvcc, sm_100a)")
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(DnTensor)
        lib.deltanet_fwd.restype = ctypes.c_int
        lib.deltanet_fwd.argtypes = [P, P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_void_p]
        lib.deltanet_fwd_ex.restype = ctypes.c_int
        lib.deltanet_fwd_ex.argtypes = [P, P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_void_p,
                                        ctypes.c_int]
        lib.gated_deltanet_fwd.restype = ctypes.c_int
        lib.gated_deltanet_fwd.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, P,
                                           ctypes.c_void_p]
        lib.gated_deltanet_fwd_ex.restype = ctypes.c_int
        lib.gated_deltanet_fwd_ex.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, P,
                                              ctypes.c_void_p, ctypes.c_int]
        lib.gated_deltaproduct_fwd.restype = ctypes.c_int
        lib.gated_deltaproduct_fwd.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, ctypes.c_int,
                                               P, P, ctypes.c_void_p]
        lib.gated_deltaproduct_fwd_ex.restype = ctypes.c_int
        lib.gated_deltaproduct_fwd_ex.argtypes = [P, P, P, P, P, P, P, ctypes.c_int,
                                                  ctypes.c_int, P, P, ctypes.c_void_p,
                                                  ctypes.c_int]
        lib.kda_fwd.restype = ctypes.c_int
        lib.kda_fwd.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_void_p]
        lib.kda_fwd_ex.restype = ctypes.c_int
        lib.kda_fwd_ex.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_void_p,
                                   ctypes.c_int]
        lib.deltanet_fwd_states.restype = ctypes.c_int
        lib.deltanet_fwd_states.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, P, P,
                                            ctypes.c_void_p, ctypes.c_int]
        lib.deltanet_fwd_noalloc.restype = ctypes.c_int
        lib.deltanet_fwd_noalloc.argtypes = [P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_void_p]
        lib.deltanet_status_string.restype = ctypes.c_char_p
        lib.deltanet_status_string.argtypes = [ctypes.c_int]
        lib.deltanet_get_error.restype = ctypes.c_int
        lib.deltanet_get_error.argtypes = [ctypes.c_void_p]
        lib.deltanet_release_workspace.restype = None
        lib.deltanet_release_workspace.argtypes = []
        lib.deltanet_last_launches.restype = ctypes.c_int
        lib.deltanet_last_launches.argtypes = []
        lib.deltanet_set_kernel_events.restype = None
        lib.deltanet_set_kernel_events.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        lib.deltanet_test_set_wait.restype = None
        lib.deltanet_test_set_wait.argtypes = [ctypes.c_ulonglong, ctypes.c_int]
        lib.deltanet_last_schedule.restype = None
        lib.deltanet_last_schedule.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                               ctypes.POINTER(ctypes.c_int)]
        # these take the descriptors' addresses as integers (see _descriptors)
        V, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.deltanet_step.argtypes = [V, V, V, V, V, I, V, V, V, V]
        lib.deltanet_scan_fwd.argtypes = [V] * 7
        lib.deltanet_scan_bwd.argtypes = [V] * 10
        lib.deltanet_scan_step.argtypes = [V] * 6
        lib.deltanet_norm_fwd.argtypes = [V, V, V, I, V, V, V, F, V, V, V]
        lib.deltanet_norm_bwd.argtypes = [V, V, V, I, V, V, V, F] + [V] * 10
        for f in (lib.deltanet_step, lib.deltanet_scan_fwd, lib.deltanet_scan_bwd,
                  lib.deltanet_scan_step, lib.deltanet_norm_fwd, lib.deltanet_norm_bwd):
            f.restype = ctypes.c_int
        lib.deltanet_norm_workspace.restype = ctypes.c_int64
        lib.deltanet_norm_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().deltanet_status_string(int(status)).decode()


_DT = {torch.float32: DN_F32, torch.bfloat16: DN_BF16, torch.int32: DN_I32}


def describe(t: Optional[torch.Tensor]) -> Optional[DnTensor]:
    """dn_tensor view of a tensor (strides in elements); None stays None."""
    if t is None:
        return None
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    d = DnTensor()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _DT[t.dtype]
    d.ndim = t.dim()
    for i in range(4):
        d.shape[i] = t.shape[i] if i < t.dim() else 0
        d.stride[i] = t.stride(i) if i < t.dim() else 0
    return d


def _ref(d: Optional[DnTensor]):
    return None if d is None else ctypes.byref(d)


def call(q, k, v, beta, initial_state, cu_seqlens, chunk_size, out, final_state, stream,
         seg_chunks: int = 0) -> int:
    """Raw call: returns the dn_status code (no exception)."""
    lib = load()
    ds = [describe(t) for t in (q, k, v, beta, initial_state, cu_seqlens, out, final_state)]
    args = [_ref(x) for x in ds[:6]] + [int(chunk_size)] + [_ref(x) for x in ds[6:]]
    if seg_chunks:
        return lib.deltanet_fwd_ex(*args, stream, int(seg_chunks))
    return lib.deltanet_fwd(*args, stream)


def call_gated(q, k, v, beta, g, initial_state, cu_seqlens, chunk_size, out, final_state,
               stream, seg_chunks: int = 0) -> int:
    """Raw Gated DeltaNet call: returns the dn_status code (no exception)."""
    lib = load()
    ds = [describe(t) for t in (q, k, v, beta, g, initial_state, cu_seqlens, out, final_state)]
    args = [_ref(x) for x in ds[:7]] + [int(chunk_size)] + [_ref(x) for x in ds[7:]]
    if seg_chunks:
        return lib.gated_deltanet_fwd_ex(*args, stream, int(seg_chunks))
    return lib.gated_deltanet_fwd(*args, stream)


def call_kda(q, k, v, beta, g, initial_state, cu_seqlens, chunk_size, out, final_state,
             stream, seg_chunks: int = 0) -> int:
    """Raw Kimi Delta Attention call: returns the dn_status code (no exception)."""
    lib = load()
    ds = [describe(t) for t in (q, k, v, beta, g, initial_state, cu_seqlens, out, final_state)]
    args = [_ref(x) for x in ds[:7]] + [int(chunk_size)] + [_ref(x) for x in ds[7:]]
    if seg_chunks:
        return lib.kda_fwd_ex(*args, stream, int(seg_chunks))
    return lib.kda_fwd(*args, stream)


def _stream_handle(device, stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def deltanet_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                 initial_state: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, chunk_size: int = 64,
                 out: Optional[torch.Tensor] = None,
                 final_state: Optional[torch.Tensor] = None,
                 output_final_state: bool = True, stream=None, seg_chunks: int = 0):
    """DeltaNet forward on CUDA tensors through the C ABI.

    Shapes: q, k [B, T, H, d_k]; v [B, T, H, d_v]; beta [B, T, H] fp32;
    initial_state [N, H, d_k, d_v] fp32 or None; cu_seqlens int32 [N+1] or None.
    Allocates ``out`` / ``final_state`` when not given.  Returns
    (out, final_state or None).  Asynchronous on ``stream`` (default: torch's
    current stream).
    """
    if not q.is_cuda:
        raise ValueError("deltanet_fwd runs on CUDA tensors only")
    B, T, H, _ = q.shape
    dk, dv = q.shape[3], v.shape[3]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    st = call(q, k, v, beta, initial_state, cu_seqlens, chunk_size, out, final_state,
              _stream_handle(q.device, stream), seg_chunks)
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state


def gated_deltanet_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                       g: torch.Tensor, initial_state: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None, chunk_size: int = 64,
                       out: Optional[torch.Tensor] = None,
                       final_state: Optional[torch.Tensor] = None,
                       output_final_state: bool = True, stream=None, seg_chunks: int = 0):
    """Gated DeltaNet forward on CUDA tensors through the C ABI.

    As ``deltanet_fwd``, plus ``g`` [B, T, H] fp32: the per-token decay as its
    natural log, g = ln a (the state update is S <- a (I - beta k^T k) S + beta k^T v).
    """
    if not q.is_cuda:
        raise ValueError("gated_deltanet_fwd runs on CUDA tensors only")
    B, T, H, _ = q.shape
    dk, dv = q.shape[3], v.shape[3]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    st = call_gated(q, k, v, beta, g, initial_state, cu_seqlens, chunk_size, out, final_state,
                    _stream_handle(q.device, stream), seg_chunks)
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state


def kda_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
            g: torch.Tensor, initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None, chunk_size: int = 64,
            out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
            output_final_state: bool = True, stream=None, seg_chunks: int = 0):
    """Kimi Delta Attention forward on CUDA tensors through the C ABI.

    As ``deltanet_fwd``, plus ``g`` [B, T, H, d_k] fp32: the decay of every key channel
    as its natural log (the state update is S <- (I - beta k^T k) Diag(a) S + beta k^T v).
    """
    if not q.is_cuda:
        raise ValueError("kda_fwd runs on CUDA tensors only")
    B, T, H, _ = q.shape
    dk, dv = q.shape[3], v.shape[3]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    st = call_kda(q, k, v, beta, g, initial_state, cu_seqlens, chunk_size, out, final_state,
                  _stream_handle(q.device, stream), seg_chunks)
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state


def chunk_state_rows(B: int, T: int, cu_seqlens: Optional[torch.Tensor] = None,
                     chunk_size: int = 64) -> int:
    """Rows of the chunk-states buffer: B * ceil(T / C) for a dense batch; for packed
    input ceil(T / C) + N, a bound on the sum of ceil(L_n / C)."""
    n_c = (T + chunk_size - 1) // chunk_size
    return B * n_c if cu_seqlens is None else n_c + cu_seqlens.numel() - 1


def deltanet_fwd_states(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                        g: Optional[torch.Tensor] = None,
                        initial_state: Optional[torch.Tensor] = None,
                        cu_seqlens: Optional[torch.Tensor] = None, chunk_size: int = 64,
                        out: Optional[torch.Tensor] = None,
                        final_state: Optional[torch.Tensor] = None,
                        chunk_states: Optional[torch.Tensor] = None, stream=None,
                        seg_chunks: int = 0):
    """DeltaNet (g None) or Gated DeltaNet forward that also returns the state
    entering every chunk: chunk_states [rows, H, d_k, d_v] fp32 with row = global
    chunk index (see ``chunk_state_rows``; allocated zeroed when not given).
    Returns (out, final_state, chunk_states)."""
    if not q.is_cuda:
        raise ValueError("deltanet_fwd_states runs on CUDA tensors only")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    if chunk_states is None:
        rows = chunk_state_rows(B, T, cu_seqlens, chunk_size)
        chunk_states = torch.zeros((rows, H, dk, dv), dtype=torch.float32, device=q.device)
    ds = [describe(t) for t in (q, k, v, beta, g, initial_state, cu_seqlens, out, final_state,
                                chunk_states)]
    args = [_ref(x) for x in ds[:7]] + [int(chunk_size)] + [_ref(x) for x in ds[7:]]
    st = load().deltanet_fwd_states(*args, _stream_handle(q.device, stream), int(seg_chunks))
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state, chunk_states


def gated_deltaproduct_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           beta: torch.Tensor, g: torch.Tensor, n_h: int,
                           initial_state: Optional[torch.Tensor] = None,
                           cu_seqlens: Optional[torch.Tensor] = None, chunk_size: int = 64,
                           out: Optional[torch.Tensor] = None,
                           final_state: Optional[torch.Tensor] = None,
                           output_final_state: bool = True, stream=None, seg_chunks: int = 0):
    """Gated Delta Product forward on CUDA tensors through the C ABI.

    q [B, T, H, d_k]; k [B, T * n_h, H, d_k], v [B, T * n_h, H, d_v] and beta
    [B, T * n_h, H] with the n_h writes of each token on consecutive rows; g
    [B, T, H] (ln a, one per token); cu_seqlens counts tokens.  Returns
    (out [B, T, H, d_v], final_state or None).
    """
    if not q.is_cuda:
        raise ValueError("gated_deltaproduct_fwd runs on CUDA tensors only")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    ds = [describe(t) for t in (q, k, v, beta, g, initial_state, cu_seqlens, out, final_state)]
    args = [_ref(x) for x in ds[:7]] + [int(n_h), int(chunk_size)] + [_ref(x) for x in ds[7:]]
    lib = load()
    stream_h = _stream_handle(q.device, stream)
    if seg_chunks:
        st = lib.gated_deltaproduct_fwd_ex(*args, stream_h, int(seg_chunks))
    else:
        st = lib.gated_deltaproduct_fwd(*args, stream_h)
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state


def deltanet_fwd_noalloc(q, k, v, beta, initial_state=None, chunk_size: int = 64, out=None,
                         final_state=None, stream=None):
    """The forward pass through the entry point that allocates no device memory
    (for callers that cannot allocate; see include/deltanet.h).  Dense bf16
    batches with d_k = d_v = 128 only.  ``out`` and ``final_state`` are allocated
    here with torch when not given: the C call itself allocates nothing."""
    B, T, H, _ = q.shape
    if out is None:
        out = torch.empty((B, T, H, v.shape[3]), dtype=q.dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((B, H, q.shape[3], v.shape[3]), dtype=torch.float32,
                                  device=q.device)
    ds = [describe(t) for t in (q, k, v, beta, initial_state, out, final_state)]
    st = load().deltanet_fwd_noalloc(*[_ref(x) for x in ds[:5]], int(chunk_size),
                                     *[_ref(x) for x in ds[5:]],
                                     _stream_handle(q.device, stream))
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))
    return out, final_state


# dn_tensor as bytes: the operators below are called once per token and layer when decoding,
# where filling ctypes structures field by field would take longer than the kernel.
_DESC = struct.Struct("@Pii8q")
assert _DESC.size == ctypes.sizeof(DnTensor)
_PAD = (0, 0, 0, 0)
_MAX_TENSORS = 16


class _Buffers(threading.local):
    """A thread's room for the descriptors of one call (the library copies what it needs
    before the call returns)."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(_DESC.size * _MAX_TENSORS)
        self.base = ctypes.addressof(self.buf)


_buffers = _Buffers()


def _descriptors(*tensors):
    """Addresses of the descriptors of the given tensors (None stays None), good until this
    thread's next call."""
    b = _buffers
    buf, base, pack, size = b.buf, b.base, _DESC.pack_into, _DESC.size
    addr, at = [], 0
    for t in tensors:
        if t is None:
            addr.append(None)
            continue
        shape = t.shape
        n = len(shape)
        dt = _DT.get(t.dtype)
        if dt is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        if n == 4:
            pack(buf, at, t.data_ptr(), dt, 4, *shape, *t.stride())
        elif 1 <= n < 4:
            pad = _PAD[n:]
            pack(buf, at, t.data_ptr(), dt, n, *shape, *pad, *t.stride(), *pad)
        else:
            raise ValueError("1 to 4 dimensions")
        addr.append(base + at)
        at += size
    return addr


_call = None


class _General:
    """In the place of csrc/dn_call.cpp where it is missing or made for another torch: every call
    goes the general way, to the same kernels."""

    def __getattr__(self, name):
        return lambda *args: None


def _short():
    """The calls that need no marshalling here (csrc/dn_call.cpp): each takes its binding's
    arguments and answers None where they want the general way below."""
    global _call
    if _call is None:
        load()
        why = "missing or made for another torch"
        module = _General()
        if _build.call_usable():
            try:
                loader = importlib.machinery.ExtensionFileLoader("dn_call", _build.CALL)
                module = importlib.util.module_from_spec(importlib.util.spec_from_loader("dn_call", loader))
                loader.exec_module(module)
            except ImportError as e:
                why, module = str(e), _General()
        if isinstance(module, _General):
            warnings.warn(f"{_build.CALL}: {why}; calls take longer without it (run "
                          "`python -m deltanet_chunkwise_delta_b200.build`)", RuntimeWarning, stacklevel=3)
        _call = module
    return _call


def _answer(r):
    if type(r) is int:
        _check(r)
    return r


_HERE = contextlib.nullcontext()
# The current stream's handle without a Stream object around it, where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda idx: torch.cuda.current_stream(idx).cuda_stream)


def _place(name, stream, lead, *others):
    """The handle of the stream of one call, and a context in which its device and stream are
    the current ones, for the allocations and the launch."""
    idx = lead.get_device() if isinstance(lead, torch.Tensor) else -1
    if idx < 0:
        raise ValueError(f"{name} runs on CUDA tensors only")
    for t in others:
        if t is not None and t.get_device() != idx:
            raise ValueError(f"{name}: tensors on {lead.device} and {t.device}")
    if stream is not None:
        if stream.device.index != idx:
            raise ValueError(f"{name}: tensors on {lead.device}, stream on {stream.device}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    here = _HERE if torch.cuda.current_device() == idx else torch.cuda.device(idx)
    return _raw_stream(idx), here


def _like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _check(st: int) -> None:
    if st != DN_OK:
        raise DeltaNetError(st, status_string(st))


def deltanet_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                  state: torch.Tensor, g: Optional[torch.Tensor] = None, n_h: int = 1,
                  slot_idx: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream=None):
    """The delta-rule recurrences for the few tokens of a decoding step, on a cache of
    states updated in place.

    q [N, T, H, d_k]; k [N, T * n_h, H, d_k], v [N, T * n_h, H, d_v] and beta [N, T * n_h, H]
    with a token's n_h writes on consecutive rows; g None (DeltaNet), [N, T, H] (Gated
    DeltaNet, Gated Delta Product) or [N, T, H, d_k] (Kimi Delta Attention), ln a in fp32;
    state [M, H, d_k, d_v] fp32; slot_idx int32 [N] names each request's row of it (-1: a
    padding request, whose rows of out are zero), None: request n uses row n.  Returns out
    [N, T, H, d_v].  Asynchronous on ``stream`` (default: torch's current stream)."""
    if stream is None:
        r = (_call or _short()).step(q, k, v, beta, state, g, n_h, slot_idx, out)
        if r is not None:
            return _answer(r)
    handle, here = _place("deltanet_step", stream, q, k, v, beta, state, g, slot_idx, out)
    with here:
        if out is None:
            out = q.new_empty((*q.shape[:3], v.shape[-1]))
        a = _descriptors(q, k, v, beta, g, state, slot_idx, out)
        _check(load().deltanet_step(*a[:5], int(n_h), *a[5:], handle))
    return out


def deltanet_scan_fwd(x: torch.Tensor, g: torch.Tensor,
                      initial_state: Optional[torch.Tensor] = None,
                      cu_seqlens: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None,
                      output_final_state: bool = True, stream=None):
    """The gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t, channel by channel.

    x [B, T, D] bf16 or fp32; g [B, T, D] fp32 (or bf16 with bf16 x), ln of the decay;
    initial_state [N, D] fp32 or None; cu_seqlens int32 [N+1] or None.  Returns (out,
    final_state or None): every h_t in the dtype of x and the last one of each sequence
    in fp32.  Outside autograd: ``deltanet_scan_bwd`` gives the gradients."""
    if stream is None:
        r = (_call or _short()).scan_fwd(x, g, initial_state, cu_seqlens, out, final_state,
                                         output_final_state)
        if r is not None:
            return _answer(r)
    handle, here = _place("deltanet_scan_fwd", stream, x, g, initial_state, cu_seqlens, out, final_state)
    with here:
        if out is None:
            out = _like(x)
        if final_state is None and output_final_state:
            n = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            final_state = torch.empty((n, x.shape[-1]), dtype=torch.float32, device=x.device)
        a = _descriptors(x, g, initial_state, cu_seqlens, out, final_state)
        _check(load().deltanet_scan_fwd(*a, handle))
    return out, final_state


def deltanet_scan_bwd(g: torch.Tensor, out: torch.Tensor, d_out: torch.Tensor,
                      initial_state: Optional[torch.Tensor] = None,
                      cu_seqlens: Optional[torch.Tensor] = None,
                      d_final_state: Optional[torch.Tensor] = None,
                      d_x: Optional[torch.Tensor] = None, d_g: Optional[torch.Tensor] = None,
                      d_initial_state: Optional[torch.Tensor] = None, stream=None):
    """Gradients of ``deltanet_scan_fwd`` from its output ``out``: (d_x, d_g,
    d_initial_state), the last where initial_state (or a buffer for it) is given, else
    None.  d_final_state [N, D] fp32, or None for zeros."""
    if stream is None:
        r = (_call or _short()).scan_bwd(g, out, d_out, initial_state, cu_seqlens, d_final_state,
                                         d_x, d_g, d_initial_state)
        if r is not None:
            return _answer(r)
    handle, here = _place("deltanet_scan_bwd", stream, g, out, d_out, initial_state, cu_seqlens,
                          d_final_state, d_x, d_g, d_initial_state)
    with here:
        if d_x is None:
            d_x = _like(out)
        if d_g is None:
            d_g = _like(g)
        if d_initial_state is None and initial_state is not None:
            d_initial_state = _like(initial_state)
        a = _descriptors(g, out, initial_state, cu_seqlens, d_out, d_final_state, d_x, d_g,
                               d_initial_state)
        _check(load().deltanet_scan_bwd(*a, handle))
    return d_x, d_g, d_initial_state


def deltanet_scan_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                       slot_idx: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream=None):
    """The gated linear recurrence for the few tokens of a decoding step: x, g [N, T, D],
    state [M, D] fp32 updated in place, slot_idx as ``deltanet_step``.  Returns out
    [N, T, D]."""
    if stream is None:
        r = (_call or _short()).scan_step(x, g, state, slot_idx, out)
        if r is not None:
            return _answer(r)
    handle, here = _place("deltanet_scan_step", stream, x, g, state, slot_idx, out)
    with here:
        if out is None:
            out = _like(x)
        a = _descriptors(x, g, state, slot_idx, out)
        _check(load().deltanet_scan_step(*a, handle))
    return out


_ACTIVATIONS = {"silu": DN_ACT_SILU, "sigmoid": DN_ACT_SIGMOID}


def _activation(name: str) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation {name!r}: one of {sorted(_ACTIVATIONS)}")
    return _ACTIVATIONS[name]


def deltanet_norm_fwd(y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None,
                      residual: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None,
                      next_weight: Optional[torch.Tensor] = None, activation: str = "silu",
                      eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                      residual_out: Optional[torch.Tensor] = None, stream=None):
    """The norms before and after a block with its gate and residual scale, over the last
    dimension d: y1 = rms_norm(y, weight), y2 = y1 activation(gate), r' = residual + scale y2,
    n = rms_norm(r', next_weight), each part where its operand is given.

    y, gate [.., d] in one dtype (bf16 or fp32); residual in that dtype or fp32; weight,
    scale, next_weight [d] fp32 or bf16; activation "silu" or "sigmoid".  Returns (out,
    residual_out): without residual (y2, None); with it (n, r'), n None without
    next_weight.  Outside autograd: ``deltanet_norm_bwd`` gives the gradients."""
    act = _activation(activation)
    if stream is None:
        r = (_call or _short()).norm_fwd(y, weight, gate, residual, scale, next_weight, act, eps,
                                         out, residual_out)
        if r is not None:
            return _answer(r)
    handle, here = _place("deltanet_norm_fwd", stream, y, weight, gate, residual, scale, next_weight,
                          out, residual_out)
    with here:
        if out is None and (residual is None or next_weight is not None):
            out = _like(y)
        if residual_out is None and residual is not None:
            residual_out = _like(residual)
        a = _descriptors(y, weight, gate, residual, scale, next_weight, out, residual_out)
        _check(load().deltanet_norm_fwd(*a[:3], act, *a[3:6], float(eps), *a[6:], handle))
    return out, residual_out


class NormGrads(NamedTuple):
    """Gradients of ``deltanet_norm_fwd``'s operands; None where one was not given.  Those of
    weight, scale and next_weight are fp32."""
    d_y: torch.Tensor
    d_weight: Optional[torch.Tensor]
    d_gate: Optional[torch.Tensor]
    d_residual: Optional[torch.Tensor]
    d_scale: Optional[torch.Tensor]
    d_next_weight: Optional[torch.Tensor]


def deltanet_norm_bwd(y: torch.Tensor, d_out: Optional[torch.Tensor],
                      weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      residual: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None,
                      next_weight: Optional[torch.Tensor] = None,
                      d_residual_out: Optional[torch.Tensor] = None, activation: str = "silu",
                      eps: float = 1e-6, stream=None, d_y: Optional[torch.Tensor] = None,
                      d_gate: Optional[torch.Tensor] = None,
                      d_residual: Optional[torch.Tensor] = None) -> NormGrads:
    """Gradients of ``deltanet_norm_fwd`` from its inputs, the gradient d_out of out (None
    where the forward call has no out) and d_residual_out of residual_out (None: zeros,
    where next_weight is given).  Buffers for the row gradients may be passed in."""
    act = _activation(activation)
    if stream is None:
        r = (_call or _short()).norm_bwd(y, d_out, weight, gate, residual, scale, next_weight,
                                         d_residual_out, act, eps, d_y, d_gate, d_residual)
        if r is not None:
            return NormGrads._make(_answer(r))
    handle, here = _place("deltanet_norm_bwd", stream, y, d_out, weight, gate, residual, scale,
                          next_weight, d_residual_out, d_y, d_gate, d_residual)
    with here:
        dev, lib = y.device, load()
        like = lambda t, given: given if given is not None or t is None else \
            torch.empty(t.shape, dtype=t.dtype, device=dev)
        d_y, d_gate, d_residual = like(y, d_y), like(gate, d_gate), like(residual, d_residual)
        params = [t is not None for t in (weight, scale, next_weight)]
        d, work, sums = y.shape[-1], None, [None] * 3
        if any(params):
            sums = [torch.empty(d, dtype=torch.float32, device=dev) if p else None for p in params]
            n = int(lib.deltanet_norm_workspace(y.numel() // d if d else 0, d))
            work = torch.empty(n, dtype=torch.float32, device=dev) if n else None
        a = _descriptors(y, weight, gate, residual, scale, next_weight, d_out,
                         d_residual_out, d_y, sums[0], d_gate, d_residual, sums[1], sums[2], work)
        _check(lib.deltanet_norm_bwd(*a[:3], act, *a[3:6], float(eps), *a[6:], handle))
    return NormGrads(d_y, sums[0], d_gate, d_residual, sums[1], sums[2])


def get_error(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) its device-side error flag."""
    return load().deltanet_get_error(_stream_handle(device, stream))


def test_set_wait(wait_ns: int = 0, stall_chunk: int = 0) -> None:
    """Test hook of the bounded device waits for the following calls on this
    thread: their time-out (0: the default 2 s) and, with stall_chunk > 0, a
    wait at chunk stall_chunk - 1 of every run that nothing completes
    (deltanet_test_set_wait in include/deltanet.h).  test_set_wait() restores
    normal calls."""
    load().deltanet_test_set_wait(int(wait_ns), int(stall_chunk))


def release_workspace() -> None:
    load().deltanet_release_workspace()


def last_launches() -> int:
    return load().deltanet_last_launches()


def set_kernel_events(start=None, stop=None) -> None:
    """Bracket the boundary-pass kernel of following calls with two
    torch.cuda.Event objects (enable_timing=True, already recorded once so that
    their handles exist); call with no arguments to stop."""
    load().deltanet_set_kernel_events(start.cuda_event if start is not None else None,
                                      stop.cuda_event if stop is not None else None)


def last_schedule(with_first: bool = False):
    """(segments per chain, chunks per segment) of the last dense call on this
    thread; with ``with_first`` also the chunks of the first segment."""
    g, s, s0 = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    load().deltanet_last_schedule(ctypes.byref(g), ctypes.byref(s), ctypes.byref(s0))
    return (g.value, s.value, s0.value) if with_first else (g.value, s.value)
