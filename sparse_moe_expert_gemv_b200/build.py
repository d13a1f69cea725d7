"""Build libmoe.so (the CUDA library) in-tree with nvcc for sm_100a, and
_marshal.so (the binding's argument marshalling for torch tensors) with g++.

Usage: python -m sparse_moe_expert_gemv_b200.build [--force] [-v]
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

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


def marshal_built_for() -> str | None:
    """The torch and Python that _marshal.so is built for: part of its binary
    interface.  None where torch or the headers it needs are not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None or shutil.which("g++") is None:
        return None
    heads = (os.path.join(os.path.dirname(spec.origin), "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(sysconfig.get_paths()["include"], "Python.h"))
    if not all(map(os.path.exists, heads)):
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # a torch that was not installed as a package
        version = f"of {os.path.getmtime(spec.origin)}"
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}"


def build_marshal(force: bool = False, verbose: bool = False) -> str | None:
    """_marshal.so, or None where it cannot be built: libmoe.so and the calls of
    the experts do without it (moe_attn_configure of the binding does not)."""
    built_for = marshal_built_for()
    if built_for is None:
        print(f"{os.path.basename(MARSHAL_SO)} is not built: it needs torch's headers, Python.h and g++",
              file=sys.stderr)
        return None
    deps = [MARSHAL_SRC, *glob.glob(os.path.join(ROOT, "include", "*.h"))]
    stamp = MARSHAL_SO + ".built_for"
    if not force and os.path.exists(MARSHAL_SO) and os.path.exists(stamp) and \
            all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL_SO) for p in deps):
        with open(stamp) as f:
            if f.read() == built_for:
                return MARSHAL_SO
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
    with open(stamp, "w") as f:
        f.write(built_for)
    return MARSHAL_SO


def build_library(force: bool = False, verbose: bool = False) -> str:
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


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_marshal(force, verbose)
    return SO


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(SO)
