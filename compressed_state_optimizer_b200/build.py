"""Build libmua.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmua.so")
SOURCES = ["mua_api.cu", "mua_select_warp.cu", "mua_apply.cu", "mua_fused.cu",
           os.path.join("muon", "muon_api.cu"), os.path.join("muon", "muon_momentum.cu"),
           os.path.join("muon", "muon_ns.cu"), os.path.join("muon", "muon_small.cu")]
HEADERS = ["mua_kernels.cuh", os.path.join("muon", "muon.cuh"),
           os.path.join("muon", "muon_tc.cuh"), os.path.join("muon", "muon_quant.cuh"), os.path.join("..", "..", "include", "mua.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    # Every fp32 operation of the bit-exact stages is an explicit _rn
    # intrinsic; no FMA contraction anywhere else either.
    "--fmad=false",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [__file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose_ptxas else []),
           "-o", tmp, *[os.path.join(CSRC, f) for f in SOURCES]]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="-v" in sys.argv)
    print(LIB)
