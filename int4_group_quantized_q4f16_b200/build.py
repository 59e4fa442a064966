"""Build the CUDA library in-tree: nvcc for sm_100a -> libzt_q4.so beside this file,
and the bounds-checked build of the same sources (-DZT_Q4_CHECKED) -> libzt_q4_checked.so.
Each source is compiled to an object of its own under build/ (only those whose sources or
headers changed, side by side) and the objects are linked.

Run ``python -m int4_group_quantized_q4f16_b200.build``.  The library links the
CUDA runtime statically, so it loads on a machine without a GPU (every entry
point that needs the device then returns an error status instead).
"""
from __future__ import annotations

import os
import subprocess
import sys
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libzt_q4.so")
LIB_CHECKED = os.path.join(PKG, "libzt_q4_checked.so")
BUILD = os.path.join(PKG, "build")
# each source with the headers of csrc/ that it includes
SOURCES = {"zt_q4.cu": ["zt_host.h", "q4_common.cuh", "q4_mma.cuh", "q4_pass.cuh", "q4_gemm_tc.cuh", "tc_common.cuh"],
           "zt_kv.cu": ["zt_host.h", "tc_common.cuh", "kv_common.cuh", "kv_cache.cuh", "kv_attn.cuh",
                        "attn_tc.cuh"],
           "zt_host.cu": ["zt_host.h"]}
NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _headers():
    return [os.path.join(INCLUDE, h) for h in os.listdir(INCLUDE) if h.endswith(".h")]


def sources():
    names = list(SOURCES) + sorted({h for hs in SOURCES.values() for h in hs})
    return [os.path.join(CSRC, n) for n in names] + _headers()


def _older(out: str, files) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in files)


def stale(lib: str = LIB) -> bool:
    return _older(lib, sources())


def build_checked(force: bool = False, verbose: bool = False) -> str:
    return build(force, verbose, LIB_CHECKED, ["-DZT_Q4_CHECKED"])


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd)


def _finish(jobs) -> None:
    bad = [p.args for p in jobs if p.wait() != 0]
    if bad:
        raise subprocess.CalledProcessError(1, bad[0])


def build(force: bool = False, verbose: bool = False, out: str = LIB, extra=()) -> str:
    if not force and not stale(out):
        return out
    os.makedirs(BUILD, exist_ok=True)
    tag = os.path.splitext(os.path.basename(out))[0]
    pid = os.getpid()
    objs, jobs, moves = [], [], []
    began = time.time()
    for src, hdrs in SOURCES.items():
        obj = os.path.join(BUILD, f"{tag}.{os.path.splitext(src)[0]}.o")
        objs.append(obj)
        if force or _older(obj, [os.path.join(CSRC, n) for n in [src, *hdrs]] + _headers()):
            tmp = f"{obj}.tmp{pid}.o"
            jobs.append(_run([_nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", "-o", tmp,
                              os.path.join(CSRC, src)], verbose))
            moves.append((tmp, obj))
    _finish(jobs)
    for tmp, obj in moves:
        os.utime(tmp, (began, began))     # a source edited while it compiled is newer than its object
        os.replace(tmp, obj)
    tmp = out + f".tmp{pid}"
    _finish([_run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], verbose)])
    os.utime(tmp, (began, began))
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
    print(build_checked(force="--force" in sys.argv, verbose=True))
