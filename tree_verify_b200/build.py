"""Build in-tree: the CUDA library tree_verify_b200/libeagle_verify.so (sm_100a only) and the Python
marshalling module tree_verify_b200/_marshal.so."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libeagle_verify.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SOURCES = [os.path.join(CSRC, "marshal.cpp"), os.path.join(ROOT, "include", "eagle_verify.h")]
SOURCES = [os.path.join(CSRC, "eagle_verify.cu")]
HEADERS = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(ROOT, "include", "eagle_verify.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v",
]


def _nvcc() -> str:
    return os.environ.get("NVCC", "nvcc")


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in sources)


def _compile(cmd, target: str, verbose: bool) -> None:
    tmp = target + f".tmp{os.getpid()}"
    res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{cmd[0]} failed to build {os.path.basename(target)}")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, target)


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale(MARSHAL, MARSHAL_SOURCES):
        return MARSHAL
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_nvcc()) or "/usr/local/cuda/bin/nvcc")))
    lib = os.path.join(base, "lib")
    _compile([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
              *(f"-isystem{d}" for d in (sysconfig.get_paths()["include"], os.path.join(base, "include"),
                                         os.path.join(cuda, "include"))),
              MARSHAL_SOURCES[0], f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
              "-lc10_cuda"], MARSHAL, verbose)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    # the library first: C programs need it where the module's compiler or headers are missing
    if force or _stale(LIB, SOURCES + HEADERS):
        _compile([_nvcc(), *NVCC_FLAGS, *SOURCES], LIB, verbose)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
