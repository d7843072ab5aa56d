"""Builds libtgdn.so (the CUDA kernels and the C ABI) in place, for sm_103a only, and
_calls.so, the part of the PyTorch binding that is C++.

Each translation unit is compiled in parallel, then linked into one shared library
beside this file (the binding into a second one).  Rebuilds only when a source or
header is newer than the libraries.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtgdn.so")
CALLS = os.path.join(HERE, "_calls.so")
BINDING = os.path.join(CSRC, "binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", f"-I{os.path.join(ROOT, 'include')}"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [BINDING] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + [os.path.join(ROOT, "include", "tgdn.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(CALLS)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    extra = list(extra or [])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    import torch
    torch_dir = os.path.dirname(torch.__file__)

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        if src == BINDING:
            include = [os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"),
                       sysconfig.get_paths()["include"],
                       os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
            run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                 f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                 *(f"-I{d}" for d in include), "-c", src, "-o", obj])
        else:
            run([NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        *objs, binding = ex.map(compile_one, [*sources(), BINDING])
    run([NVCC, *ARCH, "-shared", "-o", LIB + ".tmp", *objs])
    os.replace(LIB + ".tmp", LIB)
    libs = os.path.join(torch_dir, "lib")
    run([CXX, "-shared", "-o", CALLS + ".tmp", binding, f"-L{HERE}", "-l:libtgdn.so", f"-L{libs}",
         "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
         f"-Wl,-rpath,{libs}"])
    os.replace(CALLS + ".tmp", CALLS)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=v, extra=extra))
