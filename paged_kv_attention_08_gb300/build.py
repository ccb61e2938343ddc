"""Compile the decode library (csrc/*.cu) into ``libpa_decode.so`` for sm_103a.

Each translation unit is compiled by nvcc in parallel into ``_build/``, then
linked into a shared library beside this file.  Run ``python -m
paged_kv_attention_08_gb300.build`` (``-v`` prints ptxas register / spill /
shared-memory usage).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpa_decode.so")

SOURCES = ["pa_api.cu", "pa_step_api.cu", "pa_combine.cu", "pa_rope.cu", "pa_evict.cu",
           "pa_weights.cu", "pa_weights_tile.cu",
           "pa_attn_d64.cu", "pa_attn_d128.cu", "pa_attn_d256.cu",
           "pa_attn_d64_multi.cu", "pa_attn_d128_multi.cu", "pa_attn_d256_multi.cu",
           "pa_attn_d64_extended.cu", "pa_attn_d128_extended.cu", "pa_attn_d256_extended.cu",
           "pa_attn_d64_prefixed.cu", "pa_attn_d128_prefixed.cu", "pa_attn_d256_prefixed.cu",
           "pa_tile_d64.cu", "pa_tile_d128.cu", "pa_tile_d256.cu", "pa_tile_d256_compact.cu",
           "pa_tile_d64_extended.cu", "pa_tile_d128_extended.cu", "pa_tile_d256_extended.cu",
           "pa_tile_d256_compact_extended.cu", "pa_pair_d64.cu", "pa_pair_d128.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         f"-I{INCLUDE}"] + ARCH


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the decode library needs the CUDA toolkit to build")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pa_decode.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``libpa_decode.so`` if any source is newer; returns its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, "-shared", *ARCH, "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="-f" in sys.argv, verbose="-v" in sys.argv))
