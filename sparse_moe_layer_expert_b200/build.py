"""Build libmoefp8.so (the C-ABI CUDA library) in-tree for sm_100a.

    python sparse_moe_layer_expert_b200/build.py [--force] [--verbose]

(run by path: importing the package itself needs the built library).

Compiles every csrc/*.cu with nvcc for compute_100a/sm_100a into one shared
library next to this file.  The CUDA runtime is linked statically and the
driver API is reached through cudaGetDriverEntryPoint, so the library loads
(and exports its symbols) on a machine without a GPU driver.  csrc/binding.cpp
becomes _native.so, the Python side of the operators around the layer (torch's
own C++ headers and libraries; g++).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoefp8.so")
NATIVE = os.path.join(HERE, "_native.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(INCLUDE, "moe_fp8.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Both libraries, what is out of date of them (or all, with force)."""
    build_native(force)
    if not force and up_to_date():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
                    *objs, "-o", tmp, "-cudart", "static"], check=True)
    os.replace(tmp, LIB)
    return LIB


def _made_for() -> str:
    """What a native binding is good for: this Python's and this torch's ABI."""
    import importlib.metadata
    import sysconfig
    return f"made for {sysconfig.get_config_var('SOABI')}, torch {importlib.metadata.version('torch')}."


def native_up_to_date() -> bool:
    if not os.path.exists(NATIVE):
        return False
    t = os.path.getmtime(NATIVE)
    if any(os.path.getmtime(d) > t for d in (os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "moe_fp8.h"))):
        return False
    with open(NATIVE, "rb") as f:  # the module carries the text (MOE_MADE_FOR)
        return _made_for().encode() in f.read()


def build_native(force: bool = False) -> str:
    if not force and native_up_to_date():
        return NATIVE
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    lib = os.path.join(t, "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    subprocess.run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    f'-DMOE_MADE_FOR="{_made_for()}"', "-I", INCLUDE,
                    "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
                    "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
                    os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", lib,
                    "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib}"], check=True)
    os.replace(tmp, NATIVE)
    return NATIVE


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
