"""Build libhq.so (the C-ABI codec library) in-tree with nvcc for sm_100a.

    python -m lattice_entropy_coded_b200.build [--verbose]

Objects go to lattice_entropy_coded_b200/_build/, the library to
lattice_entropy_coded_b200/libhq.so.  A source newer than the library triggers
a rebuild of that object.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhq.so")
SOURCES = ["hq_api.cu", "hq_encode.cu", "hq_decode.cu", "hq_consume.cu", "hq_static.cu", "hq_debug.cu",
           "hq_rot_encode.cu", "hq_rot_decode.cu", "hq_haar.cu", "hq_shard.cu", "hq_rope.cu", "hq_repack.cu",
           "hq_attention.cu", "hq_attention_z.cu", "hq_attention_a2.cu", "hq_attention_d4.cu", "hq_attention_e8.cu"]
HEADERS = ["hq_internal.h", "hq_device.cuh", "hq_encode.cuh", "hq_decode.cuh", "hq_table.cuh", "hq_attention.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    # strict IEEE fp32: no contraction, no flush-to-zero, IEEE division and sqrt
    "--fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE, "-I", CSRC,
]


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    name = os.path.basename(src)
    skip = set()   # headers that few sources include
    if not name.startswith("hq_attention"):
        skip = {"hq_attention.cuh"} if name == "hq_repack.cu" else {"hq_attention.cuh", "hq_table.cuh"}
    deps = [src, os.path.join(INCLUDE, "hq.h")] + [os.path.join(CSRC, h) for h in HEADERS if h not in skip]
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, s):
            cmd = [NVCC, *NVCC_FLAGS, "-c", s, "-o", o]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(len(jobs) or 1) as ex:
        logs = list(ex.map(run, jobs))
    if verbose:
        for log in logs:
            sys.stderr.write(log)
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
