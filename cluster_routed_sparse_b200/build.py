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
FAST_SOURCE = os.path.join(CSRC, "fast_binding.cpp")
STAMP = os.path.join(PKG, "_build", "fast")
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


def _fast_stamp() -> str:
    """What _fast.so is built against besides its sources: it loads into this torch and Python only."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version}\n"


def _fast_stale() -> bool:
    if not os.path.exists(FAST) or not os.path.exists(STAMP):
        return True
    deps = [FAST_SOURCE, os.path.join(INCLUDE, "ac.h")]
    return any(os.path.getmtime(f) > os.path.getmtime(FAST) for f in deps) or open(STAMP).read() != _fast_stamp()


def _build_fast(force: bool = False) -> None:
    """fast_binding.cpp against torch's headers, linked to libac.so beside it.  Where that cannot be done (no headers,
    no compiler) the package goes without it: streaming.py makes the same calls from Python."""
    try:
        if not force and not _fast_stale():
            return
        for path in (FAST, STAMP):  # one built for another torch must not be found
            if os.path.exists(path):
                os.remove(path)
        import sysconfig

        import torch
        from torch.utils import cpp_extension

        inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
               sysconfig.get_paths()["include"], INCLUDE]
        libs = os.path.join(os.path.dirname(torch.__file__), "lib")
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in inc], FAST_SOURCE,
               "-o", FAST + ".tmp", LIB, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
               "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
        subprocess.run(cmd, check=True)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        print(f"{FAST} was not built, calls go through ctypes: {e}", file=sys.stderr)
        return
    os.replace(FAST + ".tmp", FAST)
    os.makedirs(os.path.dirname(STAMP), exist_ok=True)
    with open(STAMP, "w") as f:
        f.write(_fast_stamp())


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
    _build_fast(force)
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
