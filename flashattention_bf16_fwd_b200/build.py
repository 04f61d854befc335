"""Build in-tree: the CUDA library flashattention_bf16_fwd_b200/libfa_b200.so, and
the module _fast (csrc/fast.cpp) through which the window and cache bindings call it.

Run ``python -m flashattention_bf16_fwd_b200.build`` (or ``__graft_entry__.build()``).
nvcc cross-compiles for sm_100a; no GPU is needed to build.  The library needs
nothing else; where torch or Python's headers are missing the module is left out,
with a line on stderr (importing the bindings then says what is missing).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfa_b200.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("fa_api.cu", "fa_cache.cu", "fa_window.cu")]
HEADERS = [os.path.join(PKG, "csrc", f) for f in ("sm100.cuh", "fa_fwd.cuh", "fa_bwd.cuh", "fa_selftest.cuh",
                                                  "fa_host.h", "fa_cache.cuh", "fa_decode.cuh", "fa_window_pre.cuh")] + [
    os.path.join(ROOT, "include", f) for f in ("fa_b200.h", "fa_b200_cache.h", "fa_b200_window.h")]

FAST_SOURCE = os.path.join(PKG, "csrc", "fast.cpp")
FAST = os.path.join(PKG, "_fast" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--use_fast_math",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-cudart", "static", "--threads", "0",
]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def up_to_date(target: str = LIB, sources=()) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in sources or SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or not up_to_date():
        cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB, *SOURCES]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    build_fast(force, verbose)
    return LIB


def build_fast(force: bool = False, verbose: bool = False) -> str | None:
    """The module _fast: C++ against this interpreter's and torch's headers (None: they are not there)."""
    headers = [os.path.join(ROOT, "include", f) for f in ("fa_b200.h", "fa_b200_cache.h", "fa_b200_window.h")]
    if not force and up_to_date(FAST, [FAST_SOURCE] + headers):
        return FAST
    python = sysconfig.get_paths()["include"]
    try:
        import torch
    except ImportError as e:
        print(f"{FAST} is not built, torch is missing: {e}", file=sys.stderr)
        return None
    if not os.path.exists(os.path.join(python, "Python.h")):
        print(f"{FAST} is not built, there is no Python.h in {python}", file=sys.stderr)
        return None
    home = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), python]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in includes),
           "-o", FAST, FAST_SOURCE, "-L" + PKG, "-lfa_b200", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return FAST


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
