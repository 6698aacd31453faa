"""Build libtv.so (the CUDA kernels and their C ABI) in-tree for sm_100a.

    python -m paged_kv_cache_376_b200.build [--force] [-v]

nvcc cross-compiles without a GPU.  The library lands next to this file so
it travels with the source tree.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libtv.so")
FAST_SOURCE = os.path.join(CSRC, "fastcall.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def fast_path() -> str:
    """Where the C++ side of the binding for this torch and this interpreter
    is: it is made of both's C++, and fits no other."""
    import torch
    return os.path.join(PKG, f"_fastcall-{sysconfig.get_config_var('SOABI')}"
                             f"-torch{torch.__version__}.so")


def fast_up_to_date() -> bool:
    path = fast_path()
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in (
        FAST_SOURCE, os.path.join(INCLUDE, "tv.h"),
        os.path.join(PKG, "build.py")))


def _build_fastcall(verbose: bool = False) -> None:
    """The C++ side of _lib's ordinary calls (torch's headers, libtv's C
    calls)."""
    import torch
    path = fast_path()
    root = os.path.join(os.path.dirname(torch.__file__))
    inc = os.path.join(root, "include")
    tmp = path + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC",
           "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           os.path.join(cuda, "include"), "-isystem",
           sysconfig.get_paths()["include"], FAST_SOURCE, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", PKG, "-l:libtv.so",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_lib(force, verbose)
    if force or not fast_up_to_date():
        _build_fastcall(verbose)
    return LIB_PATH


def _build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17",
           "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC,
           "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
