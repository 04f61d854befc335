"""Build the CUDA library in-tree: flashattention_bf16_fwd_b200/libfa_b200.so.

Run ``python -m flashattention_bf16_fwd_b200.build`` (or ``__graft_entry__.build()``).
nvcc cross-compiles for sm_100a; no GPU is needed to build.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfa_b200.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("fa_api.cu", "fa_cache.cu", "fa_window.cu")]
HEADERS = [os.path.join(PKG, "csrc", f) for f in ("sm100.cuh", "fa_fwd.cuh", "fa_bwd.cuh", "fa_selftest.cuh",
                                                  "fa_host.h", "fa_cache.cuh", "fa_decode.cuh")] + [
    os.path.join(ROOT, "include", f) for f in ("fa_b200.h", "fa_b200_cache.h", "fa_b200_window.h")]

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


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB, *SOURCES]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
