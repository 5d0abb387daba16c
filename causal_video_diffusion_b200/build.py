"""Build ``libunstep.so`` (the sm_100a CUDA library behind include/unstep.h) and ``_host_calls.so``
(the native Python side of some of its calls, against torch's headers) in-tree.

``python -m causal_video_diffusion_b200.build [--force]``.  nvcc cross-compiles for sm_100a
without a GPU; the shared library links the CUDA runtime statically and needs no libcuda at link
time (the TMA descriptor encoder is fetched from the driver at run time).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libunstep.so")
# the same library with the kernels' index checks compiled in (-DUNSTEP_DEBUG): a failed check
# records UNSTEP_ERR_DEVICE_BOUNDS in the cache's error word instead of touching memory
DEBUG_LIB = os.path.join(PKG, "libunstep_debug.so")
HOST_LIB = os.path.join(PKG, "_host_calls.so")
HOST_SOURCE = os.path.join(CSRC, "host_calls.cpp")
SOURCES = ["api.cu", "rope_append.cu", "window_attn.cu", "lowrank_gemm.cu", "renoise.cu",
           "conv3d.cu", "gemm2sm.cu", "cache_q8.cu", "block_norm.cu"]
HEADERS = ["internal.h", "limits.h", "gemm.h", "conv3d.h", "sm100.cuh", "rope_append.cuh", "q8.cuh",
           "block_norm.h"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
         "--expt-relaxed-constexpr", "-Xptxas", "-v", "-I", os.path.join(ROOT, "include")]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "unstep.h"))
    return files


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    if not (force or needs_build(lib)):
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    extra = ["-DUNSTEP_DEBUG"] if debug else []
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed building {os.path.basename(lib)}")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, lib)
    return lib


def build_host(force: bool = False) -> str:
    """The extension module of csrc/host_calls.cpp; it reaches the library by addresses alone.  It
    holds for the torch and the Python that it was compiled against, and carries their names."""
    import torch
    made_for = f"host calls for torch {torch.__version__}, {sys.implementation.cache_tag}"
    inputs = [HOST_SOURCE, os.path.join(ROOT, "include", "unstep.h")]
    if not force and os.path.exists(HOST_LIB) and \
            all(os.path.getmtime(f) <= os.path.getmtime(HOST_LIB) for f in inputs):
        with open(HOST_LIB, "rb") as f:
            if made_for.encode() + b"\0" in f.read():
                return HOST_LIB
    T = os.path.dirname(torch.__file__)
    tmp = HOST_LIB + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f'-DUNSTEP_MADE_FOR="{made_for}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(T, "include"),
           "-I" + os.path.join(T, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
           "-o", tmp, HOST_SOURCE, "-L" + os.path.join(T, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(HOST_LIB)}")
    os.replace(tmp, HOST_LIB)
    return HOST_LIB


if __name__ == "__main__":
    print(build_host(force="--force" in sys.argv))
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
