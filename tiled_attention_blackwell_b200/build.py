"""Build the CUDA library ``libattn.so`` in-tree for sm_100a, and the native
part of the Python binding, ``_binding.so`` (g++, against torch's headers).

    python -m tiled_attention_blackwell_b200.build [--force]

nvcc cross-compiles without a GPU.  The CUDA runtime is linked statically, so
the library needs only the NVIDIA driver at run time.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libattn.so")
# The rescale-statistics build: the same kernels compiled with
# -DATTN_COUNT_RESCALES (per-row counters reduced into a device buffer set
# through attn_count_set_buffer); never the library the product loads.
COUNT_LIB = os.path.join(PKG, "libattn_count.so")
BINDING = os.path.join(PKG, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

# attn_api.cu: the forward and backward; sinks_*.cu: their variants with first
# keys beside a window; serve_api.cu: head norms with rotation, the paged cache
# and its decode.
UNITS = ("attn_api.cu", "sinks_fwd.cu", "sinks_parts.cu", "sinks_bwd.cu", "serve_api.cu")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "--threads", "0",
]


def _sources():
    deps = glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "attn.h"))
    return deps


def _build_one(out: str, units, defines, force: bool, verbose: bool) -> str:
    newest = max(os.path.getmtime(p) for p in _sources())
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    tmp = out + f".tmp{os.getpid()}"
    cmd = [NVCC, *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-o", tmp,
           *[os.path.join(CSRC, u) for u in units]]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the translation units (and the kernels they include) into libattn.so,
    and the binding.  Returns the library's path."""
    build_binding(force, verbose)
    return _build_one(LIB, UNITS, (), force, verbose)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/binding.cpp into _binding.so."""
    src = os.path.join(CSRC, "binding.cpp")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(ROOT, "include", "attn.h")))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest:
        return BINDING
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           "-o", tmp, src, "-L", os.path.join(base, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build_count(force: bool = False, verbose: bool = False) -> str:
    """The rescale-statistics build, libattn_count.so."""
    return _build_one(COUNT_LIB, UNITS, ("ATTN_COUNT_RESCALES",), force, verbose)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
    if "--count" in sys.argv:
        print(build_count(force="--force" in sys.argv, verbose=True))
