"""Builds libhaste.so (sm_100a) in-tree with nvcc, and with g++ the Python binding's
native argument checks, _native.<torch and Python version>.so.

The library is one translation unit (api.cu includes the kernel sources), linked
against the static CUDA runtime so that it depends only on the driver.  The argument
checks read torch's tensors by the layout of the headers that they were built with, so
their file is named after the torch, its C++ ABI and the interpreter that it is for; it is
loaded after torch, whose libraries it needs.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
OUT = os.path.join(PKG, "libhaste.so")
def _sources():
    """Every CUDA source and header of the library, and the ABI header."""
    own = [f for f in os.listdir(HERE) if f.endswith((".cu", ".cuh"))]
    return own + [os.path.join("..", "..", "include", "haste.h")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "--expt-relaxed-constexpr", "-maxrregcount=152", "-Xcompiler", "-fPIC,-O2", "-shared"]


def stale() -> bool:
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    return any(os.path.getmtime(os.path.join(HERE, s)) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        tmp = OUT + f".tmp{os.getpid()}"
        cmd = [NVCC, *FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp,
               os.path.join(HERE, "api.cu")]
        subprocess.check_call(cmd, cwd=HERE)
        os.replace(tmp, OUT)
    return OUT


NATIVE_SOURCES = [os.path.join(HERE, "native.cpp"), os.path.join(HERE, "..", "..", "include", "haste.h")]


def native_path() -> str:
    """Where the argument checks for this torch and this interpreter are, or will be, built."""
    import torch
    tag = f"torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}-{sys.implementation.cache_tag}"
    return os.path.join(PKG, f"_native.{tag}.so")


def build_native(force: bool = False) -> str:
    out = native_path()
    if not force and os.path.exists(out):
        t = os.path.getmtime(out)
        if all(os.path.getmtime(s) <= t for s in NATIVE_SOURCES):
            return out
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-o", tmp, NATIVE_SOURCES[0],
         *(a for i in include for a in ("-isystem", i)),
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-L" + os.path.join(root, "lib"),
         "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], cwd=HERE)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    build_native(force="--force" in sys.argv)
    print(OUT)
