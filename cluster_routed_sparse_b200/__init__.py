"""Cluster-routed sparse attention (AdaCluster) for one video-DiT attention
layer on NVIDIA B200 (sm_100a).

The product is libac.so, a C-ABI CUDA library (include/ac.h).  `SparseLayer`
is its thin Python binding over torch tensors; `synth` generates the seeded
synthetic inputs.  The streaming operators (rotary embedding over several axes,
attention within a window and over first tokens, the 8-bit cache) are functions
on torch tensors.  Importing the package does not load the library; the first
call does, and fails loudly if libac.so is missing.
"""

_STREAMING = ("rope_axes", "window_attn", "window_attn_backward", "Cache8", "cache8_append", "cache8_attn",
              "ops_status", "ops_check_wait_timeout")

__all__ = ["SparseLayer", "synth", *_STREAMING]


def __getattr__(name):
    if name == "SparseLayer":
        from .api import SparseLayer
        return SparseLayer
    if name in _STREAMING:
        from . import streaming
        return getattr(streaming, name)
    raise AttributeError(name)
