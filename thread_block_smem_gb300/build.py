"""Builds libswz.so in-tree (thread_block_smem_gb300/_build/) with nvcc for
sm_103a only.  Translation units compile in parallel; the library links the
CUDA runtime statically and resolves the driver's tensor-map encoder at run
time, so it loads on machines without a GPU driver (for symbol checks).

    python -m thread_block_smem_gb300.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libswz.so")
SOURCES = ["capi.cu", "transpose.cu", "gemm.cu", "l2_model.cpp", "noalloc.cu", "die.cu",
           "host_pipeline.cu", "gemm_mma_sync.cu", "tc_rate.cu", "ops.cu", "quantize.cu",
           "gemm_fp8.cu", "gemm_fp8_rows.cu", "linear_fp8.cu", "newton_schulz.cu",
           "newton_schulz_small.cu", "quantize_int8.cu", "gemm_int8.cu",
           "gemm_int8_tokens.cu", "gemm_int8_rows.cu",
           "gemm_int8_batch.cu", "layer_norm.cu",
           "layer_norm_backward.cu", "grad_norm.cu"]
HEADERS = ["common.h", "ptx.cuh", "tile_order.cuh", "ops.h", "pipe.cuh", "f8.cuh",
           "newton_schulz.cuh", "rows.cuh", "int8.cuh", "layer_norm.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (CUDA 13 toolkit required)")
    return cand


def _deps():
    return ([os.path.join(SRC_DIR, s) for s in SOURCES + HEADERS]
            + [os.path.join(ROOT, "include", "swz.h"), os.path.abspath(__file__)])


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(d) > t for d in _deps())


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    if not force and not ptxas_verbose and not _stale():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *common, "-c", os.path.join(SRC_DIR, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if ptxas_verbose or not quiet:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results],
           "-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose, quiet=False))
