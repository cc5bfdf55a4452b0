"""Compile the CUDA library (sm_100a) in-tree: libmamba_mixer.so next to this
file, and its checked build libmamba_mixer_checked.so (compiled with
MM_CHECK_BOUNDS: the forward and decode kernels check every index they form
against its buffer, skip an access outside it and report MM_ERR_BOUNDS; those of
the gated delta rule and of the 4-bit projection do not); and the Python module
of the calls a decoded token makes, _calls.so, where that can be compiled.

    python -m mamba_selective_scan_core_b200.build [--force] [--verbose] [--checked]
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
SOURCE = os.path.join(CSRC, "mixer_api.cu")
LIB_PATH = os.path.join(PKG, "libmamba_mixer.so")
CHECKED_LIB_PATH = os.path.join(PKG, "libmamba_mixer_checked.so")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
CALLS_PATH = os.path.join(PKG, "_calls.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the mixer library")


def _inputs():
    return [SOURCE] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(path: str, flags, verbose: bool) -> str:
    tmp = path + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *flags, "-I", INCLUDE, "-o", tmp, SOURCE]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)
    return path


def calls_for() -> str:
    """What the module of calls.cpp depends on besides its source: C++ of this
    torch, C of this Python.  The module holds it as a string."""
    import torch

    return f"calls.cpp for torch {torch.__version__}, {sys.implementation.cache_tag}"


def calls_fit() -> bool:
    """Is there a module of calls.cpp compiled against what runs this?"""
    try:
        with open(CALLS_PATH, "rb") as f:
            return calls_for().encode() + b"\0" in f.read()
    except OSError:
        return False


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """The module of calls.cpp, against the torch and Python that run this."""
    newest = max(os.path.getmtime(f) for f in (CALLS_SOURCE, os.path.join(INCLUDE, "mamba_mixer.h")))
    if not force and calls_fit() and os.path.getmtime(CALLS_PATH) >= newest:
        return CALLS_PATH
    if os.path.exists(CALLS_PATH):
        os.remove(CALLS_PATH)              # one that is behind its source is not loaded either
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f'-DMM_CALLS_FOR="{calls_for()}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           CALLS_SOURCE, "-o", tmp, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS_PATH)
    return CALLS_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    try:
        build_calls(force, verbose)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        # the library itself needs neither torch nor g++
        print(f"{os.path.basename(CALLS_SOURCE)} is not compiled ({e}): its calls go through ctypes", file=sys.stderr)
    if not force and not stale(LIB_PATH):
        return LIB_PATH
    return _compile(LIB_PATH, list(extra_flags), verbose)


def build_checked(force: bool = False, verbose: bool = False) -> str:
    """The checked build (index checks in the forward and decode kernels)."""
    if not force and not stale(CHECKED_LIB_PATH):
        return CHECKED_LIB_PATH
    return _compile(CHECKED_LIB_PATH, ["-DMM_CHECK_BOUNDS"], verbose)


if __name__ == "__main__":
    if "--checked" in sys.argv:
        print(build_checked(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
    else:
        print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
