"""Build libsparse_decode.so in-tree with nvcc for sm_100a, and _paged_calls.so,
the compiled form of the paged calls' Python side, with g++ against torch.

Usage: python -m token_sparse_attention_sm_b200.build [--force]"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsparse_decode.so")
CALLS = os.path.join(PKG, "_paged_calls.so")
CALLS_SRC = os.path.join(CSRC, "binding", "paged_calls.cpp")
OBJDIR = os.path.join(PKG, "_build")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
         "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newest_input():
    files = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "sparse_decode.h"),
                                                 os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def calls_tag() -> str:
    """What _paged_calls.so is compiled against, a text that the file holds:
    torch's version and C++ ABI, and the interpreter's ABI."""
    import torch
    return (f"paged_calls for torch {torch.__version__} "
            f"abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')};")


def calls_current() -> bool:
    """Whether _paged_calls.so is there and fits this torch and interpreter."""
    if not os.path.exists(CALLS):
        return False
    with open(CALLS, "rb") as f:
        return calls_tag().encode() in f.read()


def build_calls(force: bool = False) -> str:
    """_paged_calls.so: torch tensors in, the C entry points (given to it by
    address) called directly."""
    newest = max(os.path.getmtime(f) for f in
                 (CALLS_SRC, os.path.join(INCLUDE, "sparse_decode.h"), os.path.abspath(__file__)))
    if not force and calls_current() and os.path.getmtime(CALLS) >= newest:
        return CALLS
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    tmp = CALLS + f".tmp{os.getpid()}"
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-DTORCH_EXTENSION_NAME=_paged_calls", f'-DPAGED_CALLS_TAG="{calls_tag()}"', *(f"-I{p}" for p in inc), CALLS_SRC,
        f"-L{os.path.join(root, 'lib')}", "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python",
        "-o", tmp])
    os.replace(tmp, CALLS)
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)  # needs nothing of torch
    build_calls(force)
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        subprocess.check_call([NVCC, *FLAGS, *extra, "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                           *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
