"""Build libdmuon.so in-tree with hipcc for gfx950.

Usage: python -m matrix_orthogonalising_optimizer_amd.build [--jobs N]

Every translation unit under csrc/ is compiled to an object in
csrc/_build/ (in parallel), then linked into
matrix_orthogonalising_optimizer_amd/libdmuon.so.
"""

from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(CSRC, "_build")
LIB = os.path.join(PKG, "libdmuon.so")
ROOT = os.path.dirname(PKG)

ARCH = os.environ.get("DMUON_OFFLOAD_ARCH", "gfx950")
SOURCES = ["gemm_f16.hip", "gemm_bf16.hip", "gemm_f32.hip", "elementwise.hip", "small.hip", "adamw.hip", "scratch.hip", "dmuon.cpp", "owners.cpp",
           "linear_bf16_256.hip", "linear_bf16_128.hip", "linear_bf16_64.hip", "linear_f32_128.hip",
           "linear_f32_64.hip", "linear_split_256.hip",
           "norm.hip", "passes.hip", "train.cpp",
           "attention_bf16_64.hip", "attention_bf16_96.hip", "attention_bf16_128.hip", "attention_bf16_256.hip",
           "attention_f32_64.hip", "attention_f32_96.hip", "attention_f32_128.hip",
           "heads.hip", "dropout.hip", "attention.cpp"]
COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def hipcc() -> str:
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; ROCm is required to build libdmuon")
    return exe


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(jobs: int | None = None, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, os.cpu_count() or 1))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    args = ap.parse_args(argv)
    build(args.jobs, verbose=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
