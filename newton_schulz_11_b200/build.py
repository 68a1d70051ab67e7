"""Builds libmuon_b200.so in-tree with nvcc for sm_100a.

    python -m newton_schulz_11_b200.build [--verbose]

and _layers.so, the CPython module through which PyTorch tensors reach its layer entry points.

The library links the CUDA runtime statically and resolves the driver's
tensor-map encoder at run time, so it loads on machines without a GPU driver
(its entry points then report MUON_ERR_NO_DEVICE / MUON_ERR_CUDA).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from typing import List

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmuon_b200.so")
BINDING = os.path.join(PKG, "_layers.so")
BINDING_SOURCE = os.path.join(CSRC, "layers_binding.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["muon_elementwise.cu", "muon_ns_gemm.cu", "muon_host.cu", "muon_adamw.cu",
           "muon_norm.cu", "muon_linear.cu", "muon_product.cu"]
HEADERS = ["muon_device.cuh", "muon_params.h", "muon_layers.cuh", "muon_layers_host.h",
           "muon_product.h", "muon_epilogue.cuh"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmuon_b200.so")
    return cand


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "muon_b200.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(target: str, files: List[str]) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """The CPython module: host code only, linked against the library beside it."""
    if not force and _newer(BINDING, [BINDING_SOURCE, os.path.join(INCLUDE, "muon_b200.h"), os.path.abspath(__file__)]):
        return BINDING
    import sysconfig

    import torch

    base = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           BINDING_SOURCE, "-o", tmp, "-L", PKG, "-l:libmuon_b200.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda",
           "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False, force: bool = False) -> str:
    if not force and up_to_date():
        build_binding(verbose)
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(verbose, force)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
