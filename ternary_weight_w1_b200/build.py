"""Build libbitlinear.so in-tree with nvcc for sm_100a (B200).

    python -m ternary_weight_w1_b200.build        # or build() from Python

The library is one CUDA translation unit (the kernels and the C ABI) plus
the host packer and the packed-weight file reader and writer. cudart is
linked statically so the library does not depend on which CUDA runtime the
host process loaded first. Beside it stands _fastcall.so, a Python extension
that marshals the paged-cache calls (csrc/fastcall.cpp, built with g++); it is
left out where torch or its headers are missing.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbitlinear.so")
SOURCES = [os.path.join(CSRC, "bitlinear.cu"), os.path.join(CSRC, "pack.cpp"),
           os.path.join(CSRC, "packfile.cpp")]
# Everything the translation units include: every header in csrc/ and the ABI header.
DEPS = SOURCES + sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")) + [
    os.path.join(HERE, "..", "include", "bitlinear.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O3", "-Xcompiler", "-Wall,-Wextra",
    "-shared", "-cudart", "static",
]


# The C++ marshalling of the paged-cache calls, built against torch's headers.
FAST_SOURCE = os.path.join(CSRC, "fastcall.cpp")
FAST_LIB = os.path.join(HERE, "_fastcall.so")


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in DEPS if os.path.exists(d))


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    cmd = [nvcc(), *NVCC_FLAGS, *extra, *SOURCES, "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def build_fastcall(force: bool = False, verbose: bool = False) -> str | None:
    """The marshalling extension, or None without torch and its headers: the
    library needs neither, and the binding works without the extension."""
    deps = (FAST_SOURCE, os.path.join(HERE, "..", "include", "bitlinear.h"))
    if not force and os.path.exists(FAST_LIB) and all(
            os.path.getmtime(FAST_LIB) >= os.path.getmtime(d) for d in deps):
        return FAST_LIB
    import sysconfig

    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    if not os.path.isdir(os.path.join(root, "include")):
        return None
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in (f"{root}/include",
                                      f"{root}/include/torch/csrc/api/include",
                                      f"{cuda}/include", sysconfig.get_paths()["include"])),
           FAST_SOURCE, "-o", FAST_LIB + ".tmp", f"-L{root}/lib", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + r.stdout + r.stderr)
    os.replace(FAST_LIB + ".tmp", FAST_LIB)
    return FAST_LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else ())
    build_fastcall(force="--force" in sys.argv, verbose=True)
