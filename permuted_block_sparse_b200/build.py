"""Build libpbs.so (sm_100a) in-tree with nvcc.

Usage: python -m permuted_block_sparse_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpbs.so")
SOURCES = ["api.cu", "permute.cu", "permute_seg.cu", "select.cu", "select_sample.cu", "attn_fwd.cu",
           "attn_fwd_pair.cu", "permute_queries.cu",
           "permute_noalloc.cu", "cache_api.cu", "cache_attn.cu", "cache_attn_wide.cu", "key_mass.cu", "evict.cu"]
HEADERS = ["pbs_common.cuh", "pbs_internal.h", "cache_common.cuh", "cache_attn.cuh", "mma_sync.cuh", "wide_order.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _deps():
    yield os.path.join(ROOT, "include", "pbs.h")
    for h in HEADERS:
        yield os.path.join(CSRC, h)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    dep_mtime = max(os.path.getmtime(p) for p in _deps())
    objs = []
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(sp), dep_mtime)):
            continue
        cmd = [_nvcc(), *ARCH, *FLAGS, "-c", sp, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [_nvcc(), *ARCH, "-shared", "-o", LIB, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
