"""Build the CUDA library in-tree: bit_nf4_quantized_10_b200/libqlora_nf4.so.

nvcc cross-compiles for sm_100a (no GPU needed).  No fast-math: the kernels
rely on IEEE fp32 rounding, subnormals and correctly rounded division.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libqlora_nf4.so")
SOURCES = ["codebook.cu", "codec.cu", "gemm.cu", "lora_tc.cu", "smallm.cu", "mlp.cu", "fp4.cu", "fp4_gemm.cu", "adamw.cu", "gradnorm.cu", "norm.cu", "int8.cu", "trace.cu", "noalloc.cu", "diag.cu", "api.cu"]
HEADERS = ["common.cuh", "sm100.cuh", "trace.cuh"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def flags() -> list[str]:
    return ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off", "-shared", "-t", "0",
            "-I" + os.path.join(ROOT, "include")]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "qlora_nf4.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + flags() + ["-o", tmp] + [os.path.join(CSRC, f) for f in SOURCES]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
