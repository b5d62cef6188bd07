"""Builds libsp24.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_binding.so (the native half of the Python binding) with g++.  The library needs
nvcc alone; where g++, Python's or torch's CUDA headers are missing it is built
without the binding."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsp24.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-shared", "-Xcompiler", "-fPIC",
    "-Xptxas", "-v" if os.environ.get("SP24_PTXAS_VERBOSE") else "-O3",
]


def _sources():
    out = []
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(d, f))
    return out


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsp24")
    return cand


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout, res.stderr, file=sys.stderr)


def binding_tag() -> str:
    """The Python and torch that _binding.so is compiled against; it holds this text."""
    import torch
    return f"sp24 binding for {sysconfig.get_config_var('SOABI')}, torch {torch.__version__}"


def _binding_lacks() -> str:
    """What this machine lacks to compile _binding.so ("" if nothing)."""
    try:
        import torch
    except ImportError:
        return "torch"
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    if torch.version.cuda is None or not os.path.exists(
            os.path.join(inc, "c10", "cuda", "CUDAStream.h")):
        return "torch's CUDA headers"
    return ""


def needs_binding() -> bool:
    if not os.path.exists(BINDING):
        return True
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(d) > t for d in (BINDING_SRC, os.path.join(INCLUDE, "sp24.h"))):
        return True
    with open(BINDING, "rb") as f:   # of another Python or torch
        return binding_tag().encode() not in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile _binding.so (against torch's headers) unless it is up to date."""
    if not force and not needs_binding():
        return BINDING
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    lib = os.path.join(t, "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DSP24_BINDING_TAG="{binding_tag()}"',
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
          "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
          "-I", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
          "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
         verbose)
    os.replace(tmp, BINDING)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libsp24.so unless it is up to date."""
    if not force and not needs_build():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc_path(), *NVCC_FLAGS, "-I", INCLUDE, os.path.join(CSRC, "libsp24.cu"), "-o", tmp]
    _run(cmd, verbose)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libsp24.so and, where this machine can, _binding.so unless they are
    up to date; returns the library's path."""
    build_library(force, verbose)
    lacks = _binding_lacks()
    if not lacks:
        build_binding(force, verbose)
    elif lacks == "torch" or force or needs_binding():
        warnings.warn(f"_binding.so was not built, {lacks} not found: the e4m3 and norm functions "
                      "of the Python binding will raise", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
