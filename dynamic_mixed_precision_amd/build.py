"""Build libdmpq.so (the gfx950 HIP kernels and their C ABI) in-tree with hipcc.

Usage: python -m dynamic_mixed_precision_amd.build [-v]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libdmpq.so")
BUILD_DIR = os.path.join(ROOT, "_build", "dmpq")

# The GEMMs with a linear's epilogue come first: they take longest to compile.
SOURCES = ["gemm_nvfp4_linear.hip", "gemm_nvfp4_linear_lora.hip", "gemm_bf16_linear.hip", "gemm_int8_linear.hip",
           "gemm_nvfp4_linear_heads.hip", "gemm_bf16_linear_heads.hip", "gemm_int8_linear_heads.hip",
           "gemm_int8.hip", "gemm_nvfp4.hip", "gemm_bf16.hip",
           "linear_mid_bf16.hip", "linear_mid_int8.hip", "linear_mid_nvfp4.hip", "linear.hip", "qk.hip",
           "api.hip", "quant.hip", "reduce.hip", "lora.hip", "adamw.hip", "selftest.hip", "noalloc.hip"]
ARCH = "gfx950"

# -ffp-contract=off: every fp32 expression is a sequence of single IEEE RNE
#   operations, as the bit-exact quantizers require.
# -packed-fp32-ops off: no v_pk_{add,mul,fma}_f32 generation.
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the gfx950 library cannot be built")
    return path


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
