"""Build step for libfa.so: one nvcc invocation for sm_100a, output in-tree.

``build_library(debug=True)`` builds ``libfa_debug.so`` with ``-DFA_DEBUG``: the
same kernels with device-side argument checks on every TMA copy, tensor-memory
access and MMA (a failed check is reported as FA_ERR_CHECK by fa_check_status);
the Python binding loads it when the environment sets FA_DEBUG=1."""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfa.so")
LIB_DEBUG = os.path.join(PKG, "libfa_debug.so")
SOURCES = ["api.cu", "sm100.cuh", "fwd.cuh", "bwd.cuh", "fp8.cuh", "decode.cuh", "fwd256.cuh", "bwd256.cuh",
           "early.cuh", "kv4.cuh", "evict.cuh", "key_weights.cuh", "api_cache.cuh"]
CALL = os.path.join(PKG, "_fa_call.so")  # the cache operators' argument marshalling (csrc/call.cpp)
CALL_STAMP = os.path.join(PKG, "_fa_call.stamp")  # what it was built with
HEADER = os.path.join(os.path.dirname(PKG), "include", "fa.h")


def nvcc_command(out: str = LIB, extra=()):
    return [
        "nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-lineinfo",
        "-Xcompiler", "-fPIC", "-shared", "--cudart", "static", *extra,
        os.path.join(CSRC, "api.cu"), "-o", out,
    ]


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + [HEADER]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def call_command(out: str = CALL):
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(device_type="cuda")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *(f"-I{i}" for i in inc), os.path.join(CSRC, "call.cpp"), "-o", out, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]


def _call_made_with() -> str:
    import torch

    return f"torch {torch.__version__}, Python {sys.version}"


def needs_build_call() -> bool:
    deps = (os.path.join(CSRC, "call.cpp"), HEADER, os.path.abspath(__file__))
    try:
        with open(CALL_STAMP) as f:
            made_with = f.read()
        t = os.path.getmtime(CALL)
    except FileNotFoundError:
        return True
    return made_with != _call_made_with() or any(os.path.getmtime(p) > t for p in deps)


def build_call(force: bool = False) -> str:
    """_fa_call.so.  One that is out of date goes before the next is built: it passes arguments by position, and
    links against one torch."""
    made_with = _call_made_with()
    if force or needs_build_call():
        for path in (CALL_STAMP, CALL):
            if os.path.exists(path):
                os.remove(path)
        tmp = f"{CALL}.{os.getpid()}"
        subprocess.run(call_command(tmp), check=True)
        os.replace(tmp, CALL)
        with open(CALL_STAMP, "w") as f:
            f.write(made_with)
    return CALL


def build_library(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """The C library, which needs nvcc alone; then, where torch, its headers and Python's are there, the
    binding's extension module (without it the binding lacks the cache operators; build_call() says why)."""
    out = LIB_DEBUG if debug else LIB
    if force or needs_build(out):
        extra = (("-Xptxas", "-v") if verbose else ()) + (("-DFA_DEBUG",) if debug else ())
        subprocess.run(nvcc_command(out=out, extra=extra), check=True)
    try:
        build_call(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"_fa_call.so, which the cache operators' Python calls need, is not built: {e}")
    return out


if __name__ == "__main__":
    dbg = "--debug" in sys.argv
    print(build_library(force=True, verbose=True, debug=dbg))
