"""Builds the sm_100a shared library behind the C ABI (include/deltanet.h).

``python -m deltanet_chunkwise_delta_b200.build`` compiles the ``csrc/*.cu``
files with nvcc into ``_build/libdeltanet_b200.so`` inside the package directory, so
the library travels with the source tree, and ``csrc/dn_call.cpp``, the binding's short
way to it, with g++ into ``_build/dn_call.so`` beside it.  That one is made for one torch and
one Python (named in ``_build/dn_call.abi``); where it cannot be made, the binding does without.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", name)
        for name in ("deltanet.cu", "deltanet_noalloc.cu", "deltanet_ops.cu", "deltanet_norm.cu")]
LIB = os.path.join(PKG, "_build", "libdeltanet_b200.so")
CALL = os.path.join(PKG, "_build", "dn_call.so")
CALL_SRCS = [os.path.join(PKG, "csrc", "dn_call.cpp"), os.path.join(ROOT, "include", "deltanet.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
    "--threads", "0",
]


def _sources():
    return [s for s in sorted(glob.glob(os.path.join(PKG, "csrc", "*"))) if s != CALL_SRCS[0]] + \
        [os.path.join(ROOT, "include", "deltanet.h")]


def _older(path: str, sources) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(s) > os.path.getmtime(path) for s in sources)


def stale() -> bool:
    return _older(LIB, _sources())


def abi() -> str:
    """The torch and the Python that CALL has to be made for."""
    import torch
    return f"torch {torch.__version__} {sys.implementation.cache_tag}"


def call_usable() -> bool:
    """CALL is there and made for this torch and this Python."""
    if not os.path.exists(CALL):
        return False
    try:
        with open(CALL[:-3] + ".abi") as f:
            return f.read() == abi()
    except OSError:
        return False


def _run(cmd, verbose):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stderr)
    return res.stderr


def _build_call(verbose: bool) -> None:
    """The binding's short way: linked to the library beside it and to torch's own."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = CALL + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
          "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include"),
          "-isystem", sysconfig.get_paths()["include"], "-o", tmp,
          os.path.join(PKG, "csrc", "dn_call.cpp"), "-L" + os.path.dirname(LIB),
          "-l:" + os.path.basename(LIB), "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda",
          "-ltorch", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, CALL)
    with open(CALL[:-3] + ".abi", "w") as f:
        f.write(abi())


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    if force or stale():
        _build_lib(verbose)
    if force or _older(CALL, CALL_SRCS) or not call_usable():
        try:
            _build_call(verbose)
        except (OSError, RuntimeError) as e:    # no g++, no Python headers: the calls go through ctypes
            if os.path.exists(CALL):
                os.remove(CALL)
            sys.stderr.write(f"{CALL} was not built, calls take longer without it: {e}\n")
    return LIB


def _build_lib(verbose: bool) -> None:
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-o", tmp, *SRCS]
    err = _run(cmd, verbose)
    log = os.path.join(os.path.dirname(LIB), "ptxas.log")
    with open(log, "w") as f:
        f.write(err)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
