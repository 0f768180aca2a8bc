"""Builds libkda.so (the CUDA library behind include/kda.h) in-tree with nvcc
for sm_100a.  Usage: ``python -m kimi_delta_attention_31_b200.build [--force]``."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libkda.so")
CSRC = os.path.join(PKG, "csrc")
UNITS = [os.path.join(CSRC, "kda_api.cu"), os.path.join(CSRC, "kda_layer_api.cu")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    # without unique symbols: two copies of the library in one process would share
    # which kernels have been set up, and the second copy's never would be
    "-Xcompiler", "-fPIC,-fno-gnu-unique",
    "-Xptxas", "-warn-spills",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "kda.h")])


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not needs_build():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    objects = [f"{tmp}.{i}.o" for i in range(len(UNITS))]
    compiles = [[nvcc, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", "-o", o, u]
                for o, u in zip(objects, UNITS)]
    try:
        running = []
        for cmd in compiles:
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd))
        codes = [p.wait() for p in running]
        for cmd, code in zip(compiles, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.run([nvcc, *NVCC_FLAGS[:2], "-shared", "-o", tmp, *objects], check=True)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force or bool(extra), verbose=True, extra=extra))
