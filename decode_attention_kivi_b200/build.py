"""Builds libkivi.so (the C ABI of include/kivi.h) in-tree for sm_100a with nvcc, and
_kivi_torch.so (the tensor checks and calls of the paged-cache binding) with g++."""
from __future__ import annotations

import importlib.metadata
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkivi.so")
BINDING = os.path.join(PKG, "_kivi_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "kivi_torch.cpp")
BINDING_TARGET = os.path.join(PKG, "_build", "binding_target")  # what the binding was built for
DEBUG_LIB = os.path.join(PKG, "libkivi_debug.so")
# debug build: short bounded waits (about 1 ms), copy bounds checks, a test hook
DEBUG_FLAGS = ["-DKIVI_DEBUG_BUILD", "-DKIVI_DEBUG_BOUNDS", "-DKIVI_DEBUG_WAIT_CYCLES=2000000LL"]
SOURCES = ["kivi_api.cu", "kivi_quant.cu", "kivi_attn.cu", "kivi_bf16_attn.cu",
           "kivi_prefill_attn.cu", "kivi_paged_api.cu", "kivi_paged.cu", "kivi_paged_decode.cu",
           "kivi_varlen_attn.cu"]
NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-warn-spills",
]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".h"))]
    return files + [os.path.join(ROOT, "include", "kivi.h")]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in _inputs())


def binding_target() -> str:
    """The torch and the Python that a binding is built for: their interfaces change by release."""
    return f"torch {importlib.metadata.version('torch')}, Python {sysconfig.get_python_version()}"


def binding_stale() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_TARGET):
        return True
    with open(BINDING_TARGET) as f:
        if f.read() != binding_target():
            return True
    inputs = [BINDING_SOURCE, os.path.join(ROOT, "include", "kivi.h")]
    return any(os.path.getmtime(f) > os.path.getmtime(BINDING) for f in inputs)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Builds _kivi_torch.so against the torch that is installed, when stale."""
    if not force and not binding_stale():
        return BINDING
    import torch
    from torch.utils.cpp_extension import include_paths
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    dirs = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DKIVI_BINDING_TARGET="{binding_target()}"',
           *[f"-I{d}" for d in dirs], BINDING_SOURCE, "-o", tmp,
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_TARGET), exist_ok=True)
    with open(BINDING_TARGET, "w") as f:
        f.write(binding_target())
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Builds libkivi.so (or, with debug=True, libkivi_debug.so) and the binding when stale."""
    build_binding(force and not debug, verbose)
    lib = DEBUG_LIB if debug else LIB
    if not force and not stale(lib):
        return lib
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = lib + ".tmp"
    cmd = [nvcc, *NVCC_FLAGS, *(DEBUG_FLAGS if debug else []), "-o", tmp,
           *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
