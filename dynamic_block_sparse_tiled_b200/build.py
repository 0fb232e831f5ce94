"""Build the in-tree CUDA library ``libblasst.so`` for sm_100a with nvcc.

Usage: ``python -m dynamic_block_sparse_tiled_b200.build`` (or
``__graft_entry__.build()``). The shared object lands next to this file so it
travels with the source tree; it statically links the CUDA runtime.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libblasst.so")
UNITS = [os.path.join(CSRC, "blasst_capi.cu"), os.path.join(CSRC, "blasst_seq_capi.cu")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    # the units are compiled side by side, then linked
    objs = [os.path.join(PKG, os.path.basename(u) + f".{os.getpid()}.o") for u in UNITS]
    tmp = LIB + f".tmp{os.getpid()}"
    try:
        running = []
        for unit, obj in zip(UNITS, objs):
            cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, unit]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), file=sys.stderr)
            running.append((cmd, subprocess.Popen(cmd)))
        codes = [(cmd, p.wait()) for cmd, p in running]
        for cmd, rc in codes:
            if rc != 0:
                raise subprocess.CalledProcessError(rc, cmd)
        subprocess.check_call([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    finally:
        for f in objs + [tmp]:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
