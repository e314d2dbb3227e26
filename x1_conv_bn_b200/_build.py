"""Builds the in-tree shared library libx1cb.so for sm_100a with nvcc, and the
binding's marshalling module _x1cb_torch.so (C++ against torch) beside it."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libx1cb.so")
HEADER = os.path.join(HERE, "..", "include", "x1cb.h")
BINDING_SRC = os.path.join(CSRC, "x1cb_torch.cpp")
BINDING = os.path.join(HERE, "_x1cb_torch.so")
NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v", "--threads", "0",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        HEADER]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_binding(force)
    return LIB


def _built_for() -> str:
    """What the marshalling module depends on besides its sources; it holds this text."""
    import torch

    return f"_x1cb_torch for torch {torch.__version__} and {sys.implementation.cache_tag}"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    if not all(os.path.getmtime(p) <= t for p in (BINDING_SRC, HEADER)):
        return False
    with open(BINDING, "rb") as f:
        return _built_for().encode() + b"\0" in f.read()


def build_binding(force: bool = False) -> str:
    """The marshalling module: g++ against torch's headers and libx1cb.so."""
    if not force and binding_up_to_date():
        return BINDING
    import torch

    root = os.path.dirname(torch.__file__)
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc"))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if nvcc else "/usr/local/cuda"
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DX1CB_BUILT_FOR="{_built_for()}"',
           f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include",
           f"-I{cuda}/include", f"-I{sysconfig.get_paths()['include']}", BINDING_SRC, "-o", tmp,
           f"-L{root}/lib", f"-L{HERE}", "-l:libx1cb.so", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _x1cb_torch.so")
    os.replace(tmp, BINDING)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + ".tmp"
    cmd = [nvcc] + NVCC_FLAGS + ["-o", tmp] + sources()
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libx1cb.so")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, LIB)
    with open(os.path.join(HERE, "ptxas_info.txt"), "w") as f:
        f.write(res.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
