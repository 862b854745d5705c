"""Compile libfarn.so (the C ABI of include/farn.h) for sm_103a, in tree, one
process per source file."""
from __future__ import annotations

import os
import subprocess
import tempfile
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libfarn.so")
SOURCES = [os.path.join(CSRC, f) for f in
           ("farn.cu", "farn_route.cu", "farn_nvfp4.cu", "farn_product.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in
                     ("farn_kernels.cuh", "farn_internal.h", "farn_product.cuh", "farn_product_tc.cuh",
                      "farn_tcgen05.cuh")] + \
    [os.path.join(INCLUDE, "farn.h")]
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    # IEEE division and square root, denormals kept: the per-row rstd and
    # every bf16 rounding follow IEEE fp32 (no -use_fast_math, no -ftz).
    "-prec-div=true", "-prec-sqrt=true", "-ftz=false",
    "-Xcompiler", "-fPIC",
]
_lock = threading.Lock()


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in DEPENDS)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build libfarn.so next to this file if missing or older than its sources."""
    with _lock:
        if force or _stale():
            with tempfile.TemporaryDirectory(prefix="_build", dir=PKG) as d:
                def compile_one(src):
                    obj = os.path.join(d, os.path.basename(src) + ".o")
                    cmd = ["nvcc", *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src]
                    if verbose:
                        cmd.insert(1, "-Xptxas=-v")
                    subprocess.run(cmd, check=True)
                    return obj
                with ThreadPoolExecutor(len(SOURCES)) as ex:
                    objects = list(ex.map(compile_one, SOURCES))
                tmp = os.path.join(d, "libfarn.so")
                subprocess.run(["nvcc", *NVCC_FLAGS, "-shared", "-o", tmp, *objects], check=True)
                os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True))
