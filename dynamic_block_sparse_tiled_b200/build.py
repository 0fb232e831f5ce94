"""Build the in-tree CUDA library ``libblasst.so`` for sm_100a with nvcc, and
the torch binding ``_seq_binding.so`` of the sequence operators with the host
compiler.

Usage: ``python -m dynamic_block_sparse_tiled_b200.build`` (or
``__graft_entry__.build()``). The shared objects land next to this file so they
travel with the source tree; the library statically links the CUDA runtime, the
binding links the library beside it and torch's own libraries.
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
BINDING = os.path.join(PKG, "_seq_binding.so")
BINDING_UNIT = os.path.join(CSRC, "seq_binding.cpp")

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


def _binding_cmds(obj: str, out: str, lib: str):
    """Compile and link commands of the torch binding."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cxx = shutil.which("g++") or "g++"
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           os.path.join(ROOT, "include")]
    libs = cpp_extension.library_paths()
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
             *[a for d in inc for a in ("-isystem", d)], "-c", "-o", obj, BINDING_UNIT],
            [cxx, "-shared", "-o", out, obj, lib, "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in libs],
             "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda"])


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h"))


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _older(target, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def needs_build() -> bool:
    return _older(LIB, _sources()) or _older(BINDING, [BINDING_UNIT, *_headers()])


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tag = f".{os.getpid()}"
    commands, links, made = [], [], []

    def obj_of(unit):
        made.append(os.path.join(PKG, os.path.basename(unit) + tag + ".o"))
        return made[-1]

    def out_of(target):
        made.append(target + ".tmp" + tag)
        return made[-1]

    if force or _older(LIB, _sources()):
        objs = []
        for unit in UNITS:
            objs.append(obj_of(unit))
            commands.append([_nvcc(), *(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, "-I",
                             os.path.join(ROOT, "include"), "-c", "-o", objs[-1], unit])
        tmp = out_of(LIB)
        links.append(([_nvcc(), *NVCC_FLAGS, "-Xlinker", "-soname=libblasst.so", "-shared", "-o", tmp,
                       *objs], tmp, LIB))
    if force or _older(BINDING, [BINDING_UNIT, *_headers()]):
        tmp = out_of(BINDING)
        compile_cmd, link_cmd = _binding_cmds(obj_of(BINDING_UNIT), tmp, LIB)
        commands.append(compile_cmd)
        links.append((link_cmd, tmp, BINDING))
    try:
        # the units are compiled side by side, then linked (the library first)
        running = []
        for cmd in commands:
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            running.append((cmd, subprocess.Popen(cmd)))
        codes = [(cmd, p.wait()) for cmd, p in running]
        for cmd, rc in codes:
            if rc != 0:
                raise subprocess.CalledProcessError(rc, cmd)
        for cmd, tmp, target in links:
            subprocess.check_call(cmd)
            os.replace(tmp, target)
    finally:
        for f in made:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
