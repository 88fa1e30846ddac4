"""Build libthinkv.so in-tree with nvcc for sm_100a.

    python -m mixed_precision_paged_thinkv_b200.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libthinkv.so")
SOURCES = ["thinkv_api.cu", "thinkv_append.cu", "thinkv_evict.cu", "thinkv_decode.cu",
           "thinkv_noalloc.cu", "thinkv_classify.cu", "thinkv_tbe.cu",
           "thinkv_compact.cu", "thinkv_victims.cu", "thinkv_turnover.cu",
           "thinkv_shared.cu", "thinkv_prefix.cu"]
HEADERS = ["thinkv_common.cuh", "thinkv_internal.h", "thinkv_evict_seq.cuh", "thinkv_pages.cuh",
           "thinkv_shared.h"]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "thinkv.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every CUDA source and link libthinkv.so next to this file."""
    if not force and not _stale():
        return LIB
    out_dir = os.path.join(PKG, "_build")
    os.makedirs(out_dir, exist_ok=True)
    objs, jobs = [], []
    flags = NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        flags = flags + ["-Xptxas", "-v"]
    for src in SOURCES:
        obj = os.path.join(out_dir, src.replace(".cu", ".o"))
        cmd = [nvcc()] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((cmd, subprocess.Popen(cmd)))      # the sources compile side by side
        objs.append(obj)
    codes = [job.wait() for _, job in jobs]
    for (cmd, _), code in zip(jobs, codes):
        if code != 0:
            raise subprocess.CalledProcessError(code, cmd)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp] + objs + ["-lcudart"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
