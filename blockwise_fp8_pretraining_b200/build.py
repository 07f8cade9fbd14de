"""Build the CUDA library in-tree: libfp8blk.so next to this file, and the
binding's compiled host side for the installed torch beside it.

    python -m blockwise_fp8_pretraining_b200.build [--force]

Compiles csrc/fp8blk.cu for sm_100a only, and csrc/host.cpp with g++.  IEEE division, square root and
denormals are kept (no fast-math, no flush-to-zero): the quantizer's
bit-exact definition depends on them.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8blk.so")
SOURCES = [os.path.join(CSRC, f) for f in ("fp8blk.cu", "gemm.cuh", "quantize.cuh", "ptx.cuh", "swiglu.cuh", "rmsnorm.cuh",
                                              "addnorm.cuh", "logprobs.cuh", "newton_schulz.cuh",
                                              "newton_schulz_small.cuh")]
HOST_SOURCE = os.path.join(CSRC, "host.cpp")
# (its name says which torch and Python it was built for)
HOST_LIB = os.path.join(HERE, f"_fp8blk_host.torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")
HEADER = os.path.join(os.path.dirname(HERE), "include", "fp8blk.h")

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in SOURCES + [HEADER] if os.path.exists(s))


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *NVCC_FLAGS, "-o", tmp, os.path.join(CSRC, "fp8blk.cu")]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    try:
        build_host(force)
    except (OSError, subprocess.CalledProcessError) as e:      # no g++, or no headers: the binding does without
        if os.path.exists(HOST_LIB):
            os.remove(HOST_LIB)        # (of an older header, perhaps with other arguments)
        print(f"the binding's compiled host side was not built, its Python one serves: {e}", file=sys.stderr)
    return LIB


def build_host(force: bool = False) -> str:
    if not force and os.path.exists(HOST_LIB) and os.path.getmtime(HOST_LIB) >= max(map(os.path.getmtime, (HOST_SOURCE, HEADER))):
        return HOST_LIB
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    tmp = HOST_LIB + f".tmp{os.getpid()}"
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        *(f"-I{d}" for d in (sysconfig.get_paths()["include"], os.path.join(root, "include"),
                             os.path.join(root, "include", "torch", "csrc", "api", "include"),
                             os.path.join(cuda, "include"))),
        "-o", tmp, HOST_SOURCE, f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
        "-ltorch_python",
    ])
    os.replace(tmp, HOST_LIB)
    return HOST_LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
