"""Build libwkv7.so in-tree with nvcc for sm_100a (no GPU needed)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libwkv7.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    mtime = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > mtime for s in _sources())


# Translation units: the WKV7 kernels share one __device__ status word and are
# compiled together; the state-space mixer's files stand alone.
UNITS = ("libwkv7.cu", "act8.cu", "rmsnorm.cu", "conv.cu", "ssm_scan.cu", "ssm_bwd.cu")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    flags = NVCC_FLAGS + (["-Xptxas=-v"] if verbose else []) + ["-I", INCLUDE, "-I", CSRC]
    with tempfile.TemporaryDirectory() as objects:
        def unit(name):
            obj = os.path.join(objects, name + ".o")
            subprocess.check_call([NVCC, *flags, "-c", os.path.join(CSRC, name), "-o", obj])
            return obj

        with ThreadPoolExecutor(len(UNITS)) as pool:
            objs = list(pool.map(unit, UNITS))
        subprocess.check_call([NVCC, *NVCC_FLAGS, "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
