"""Build libac.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and
_fast.so, the compiled part of the Python binding, with the host compiler.

    python -m cluster_routed_sparse_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libac.so")
FAST = os.path.join(PKG, "_fast.so")
SOURCES = ["ac_api.cu", "cluster_kernels.cu", "assign_mma.cu", "score_kernels.cu", "quest_mma.cu", "attn_kernel.cu",
           "noalloc.cu", "stream_api.cu", "rope_axes.cu", "cache8.cu", "window_attn.cu",
           "window_few.cu", "window_bwd.cu"]
HEADERS = ["ac_device.cuh", "ac_internal.h", "stream_device.cuh", "stream_internal.h", "stream_host.h"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for p in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if p and (os.path.isabs(p) and os.path.exists(p) or not os.path.isabs(p)):
            return p
    return "nvcc"


def _build_fast() -> None:
    """fast_binding.cpp against torch's headers, linked to libac.so beside it."""
    import sysconfig

    from torch.utils import cpp_extension

    src = os.path.join(CSRC, "fast_binding.cpp")
    if os.path.exists(FAST) and os.path.getmtime(FAST) > max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "ac.h"))):
        return
    import torch
    inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in inc], src,
           "-o", FAST + ".tmp", LIB, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    subprocess.run(cmd, check=True)
    os.replace(FAST + ".tmp", FAST)


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "ac.h")]
    return any(os.path.getmtime(f) > t for f in deps)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every CUDA source into one shared library next to this file."""
    if not force and not _stale():
        _build_fast()
        return LIB
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--threads", "0", "-shared", "-Xlinker", "-soname=libac.so",
           "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC,
           "-o", LIB + ".tmp"] + [os.path.join(CSRC, f) for f in SOURCES] + ["-lcudart"]
    if ptxas_verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    _build_fast()
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
