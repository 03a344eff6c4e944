"""Build libmoe_b200.so from csrc/*.cu with nvcc for sm_100a (B200), and the native part of the
binding, moe_binding.so, from csrc/binding.cpp with g++ against torch's headers, in-tree.

Usage: python -m deterministic_invariant_routing_b200.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

from ._native import BINDING_PATH, binding_built_for, binding_target

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe_b200.so")
HEADER = os.path.join(ROOT, "include", "moe.h")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-Xcompiler", "-Wall",
                     "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libmoe_b200")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_up_to_date() -> bool:
    if not os.path.exists(BINDING_PATH) or binding_built_for() != binding_target():
        return False
    t = os.path.getmtime(BINDING_PATH)
    return all(os.path.getmtime(p) <= t for p in (BINDING_SRC, HEADER))


def _refresh_binding(force: bool = False) -> None:
    """Build the binding if it is out of date. It is a torch extension: without torch there is
    nothing to bind, and the library, which needs nvcc alone, stands by itself."""
    if importlib.util.find_spec("torch") is None:
        sys.stderr.write("torch not found: libmoe_b200.so is built without moe_binding.so\n")
    elif force or not _binding_up_to_date():
        _build_binding()


def _build_binding() -> None:
    import sysconfig

    import torch
    cxx = shutil.which("g++")
    if cxx is None:
        raise RuntimeError("g++ not found: it is needed to build moe_binding.so")
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = [os.path.join(os.path.dirname(torch.__file__), "include"),
           os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "api",
                        "include"),
           sysconfig.get_paths()["include"], cuda, os.path.join(ROOT, "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMOE_BINDING_TARGET="{binding_target()}"',
           *[f for d in inc for f in ("-isystem", d)], BINDING_SRC, "-o", tmp, "-L", LIB_DIR,
           "-l:libmoe_b200.so", "-L", libs, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every kernel for sm_100a and link the shared library, then the binding (where torch
    is installed). Returns the library's path."""
    if not force and not verbose_ptxas and up_to_date():
        _refresh_binding()
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), sources()))
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt",
           "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _refresh_binding(force)
    return LIB_PATH


if __name__ == "__main__":
    p = build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv)
    print(p)
