"""Builds libddl.so in-tree for sm_103a (nvcc, no CMake).

Sources compile in parallel into ``_build/``; the shared library lands next to
this file, where the binding loads it.  No fast-math: the all-reduce kernels' adds
and multiplies must be single IEEE operations.
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
OUT = os.path.join(HERE, "libddl.so")
BUILD = os.path.join(ROOT, "_build", "ddl")

SOURCES = ["plan.cpp", "ddl_api.cu", "fold_kernels.cu", "step_kernels.cu", "noalloc.cu", "sgd_kernels.cu",
           "product_kernels.cu", "product_selftest.cu", "linear_kernels.cu", "linear_api.cu", "ortho_kernels.cu",
           "ortho_api.cu"]
# contractions with no bit-exact contract: fused multiply-adds allowed
FMA_SOURCES = {"product_kernels.cu", "product_selftest.cu", "linear_kernels.cu", "ortho_kernels.cu"}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-fPIC,-Wall",
         "-I", INCLUDE, "-I", CSRC]


def _inputs():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return deps + [os.path.join(INCLUDE, "ddl.h")]


def _stale() -> bool:
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    flags = [f for f in FLAGS if f != "-fmad=false"] if src in FMA_SOURCES else FLAGS
    cmd = ["nvcc", *ARCH, *flags, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd.insert(1, "-x")
        cmd.insert(2, "c++")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not _stale():
        return OUT
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = OUT + f".tmp{os.getpid()}"
    subprocess.check_call(["nvcc", *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas" in sys.argv))
