"""Build libxp.so in-tree from csrc/*.cu for sm_103a (nvcc, no cmake)."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libxp.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

SOURCES = ["xp_api.cu", "xp_p2p.cu", "xp_p2p_tma.cu", "xp_ll.cu", "xp_ll128.cu", "xp_ring.cu", "xp_ring_tma.cu",
           "xp_noalloc.cu", "xp_proxy.cu", "xp_train.cu", "xp_adamw.cu", "xp_layernorm.cu",
           "xp_model.cu", "xp_block8.cu", "xp_matmul8.cu", "xp_rmsnorm.cu", "xp_distill.cu"]
HEADERS = ["xp_internal.h", "xp_device.cuh", "xp_proxy.h", "xp_train_internal.h", "xp_train_device.cuh", "xp_checks.h",
           "xp_model_internal.h", "xp_scales.h", "xp_code8.cuh", "xp_fours.cuh", "xp_tcgen05.cuh"]

# --fmad=false and the default -ftz=false keep the ring's fp32 adds plain IEEE
# round-to-nearest-even additions (the reductions must match the oracle bit
# for bit).
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-I", INCLUDE,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps += [os.path.join(INCLUDE, h) for h in ("xp.h", "xp_train.h", "xp_model.h")] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libxp.so next to this file; returns its path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-Xcompiler", "-fPIC",
           "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
