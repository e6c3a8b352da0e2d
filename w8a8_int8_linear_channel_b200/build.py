"""Build libsq.so (the C-ABI library) in-tree for sm_100a with nvcc.

    python w8a8_int8_linear_channel_b200/build.py [--force] [-v]

Objects go to _build/ at the repository root; the shared library lands next
to this file so the Python binding finds it.  The CUDA runtime is linked
statically and the driver's tensor-map encoder is resolved at run time, so
the library loads on a machine without a GPU driver (only calls need one).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-fmad=false",
                "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]

SOURCES = ["sq_api.cu", "k_rows.cu", "k_cols.cu", "k_gemm_tiled.cu", "k_gemm_pair.cu", "k_gemm_splitk.cu",
           "sq_api_w4.cu", "k_w4_weight.cu", "k_w4_stream.cu", "k_w4_gemm.cu", "k_moe.cu"]
HEADERS = ["sq_internal.h", "sq_ptx.cuh", "sq_tmap.h", "sq_w4.h", "sq_w4.cuh"]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + \
        [os.path.join(ROOT, "include", "sq.h")]
    if _newer(obj, deps):
        return obj
    cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel for sm_100a and link libsq.so; return its path."""
    os.makedirs(OBJDIR, exist_ok=True)
    if force:
        for s in SOURCES:
            o = os.path.join(OBJDIR, os.path.splitext(s)[0] + ".o")
            if os.path.exists(o):
                os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    if not _newer(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
