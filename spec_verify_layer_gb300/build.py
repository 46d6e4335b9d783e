"""Compiles libmoeverify.so in place for sm_103a (nvcc, one -gencode, no cmake)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("moe_verify.cu", "moe_prefill.cu", "moe_round_map.cu", "moe_qk_rope.cu",
                                                  "moe_tree_attn.cu", "moe_logprob.cu", "moe_host.cpp")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in ("moe_internal.h", "moe_common.cuh", "moe_round_ops.cuh")] + [
    os.path.join(ROOT, "include", "moe_verify.h")]
OUT = os.path.join(HERE, "libmoeverify.so")

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "--threads", "0"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(p) <= t for p in SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SOURCES]
    subprocess.check_call(cmd, cwd=HERE)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
