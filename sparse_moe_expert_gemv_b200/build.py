"""Build libmoe.so (the CUDA library) in-tree with nvcc for sm_100a, and
_marshal.so (the binding's argument marshalling for torch tensors) with g++.

Usage: python -m sparse_moe_expert_gemv_b200.build [--force] [-v]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SO = os.path.join(PKG, "libmoe.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL_SO = os.path.join(PKG, "_marshal.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def needs_build() -> bool:
    if not os.path.exists(SO):
        return True
    t = os.path.getmtime(SO)
    return any(os.path.getmtime(p) > t for p in _deps())


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    deps = [MARSHAL_SRC, *glob.glob(os.path.join(ROOT, "include", "*.h"))]
    if not force and os.path.exists(MARSHAL_SO) and \
            all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL_SO) for p in deps):
        return MARSHAL_SO
    import sysconfig

    import torch
    tp = os.path.dirname(torch.__file__)
    inc = [os.path.join(tp, "include"), os.path.join(tp, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    tmp = MARSHAL_SO + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in inc), "-o", tmp, MARSHAL_SRC, "-L" + os.path.join(tp, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, MARSHAL_SO)
    return MARSHAL_SO


def build(force: bool = False, verbose: bool = False) -> str:
    build_marshal(force, verbose)
    if not force and not needs_build():
        return SO
    tmp = SO + f".tmp{os.getpid()}"
    cmd = [NVCC, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas")
        cmd.insert(2, "-v")
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(SO)
