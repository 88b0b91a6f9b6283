"""Build libdwkv.so (the C-ABI library) in-tree for sm_100a with nvcc.

Usage: python -m decode_attention_depthweave_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libdwkv.so")
SOURCES = ["dwkv_api.cu", "dwkv_basis.cu", "dwkv_cache.cu", "dwkv_control.cu", "dwkv_decode_b4.cu", "dwkv_decode_b4p.cu",
           "dwkv_decode_b8.cu", "dwkv_decode_b8p.cu", "dwkv_decode_b4c8.cu", "dwkv_decode_b4pc8.cu",
           "dwkv_decode_b8c8.cu", "dwkv_decode_b8pc8.cu", "dwkv_nibble_api.cu", "dwkv_nibble_store.cu",
           "dwkv_nibble_attend.cu"]
HEADERS = ["dwkv_common.cuh", "dwkv_decode.cuh", "dwkv_encode.cuh", "dwkv_stored.cuh", "dwkv_nibble.cuh", "dwkv_nibble_decode.cuh", "dwkv_nibble_chunk.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-static-global-template-stub=false", "-I", INCLUDE, "-I", CSRC]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "dwkv.h")]
    if _stale(obj, deps + [__file__]):
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        subprocess.run(cmd, check=True)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if force:
        for f in os.listdir(OUT_DIR):
            if f.endswith(".o"):
                os.remove(os.path.join(OUT_DIR, f))
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
