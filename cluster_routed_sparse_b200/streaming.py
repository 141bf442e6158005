"""Streaming operators over torch tensors: what surrounds the attention of a
video generator that works frame after frame.

    rope_axes               rotary embedding over several axes, and its inverse
    window_attn             attention within a window and over a few first tokens
    window_attn_backward    its gradients
    Cache8, cache8_append, cache8_attn
                            a paged cache of keys and values in 8 bits, and the
                            attention that reads it
    ops_status              waits, and raises what the kernels have noted
    ops_check_wait_timeout  health check of that: a wait that runs out

Each call forwards data pointers, strides and the current stream of the
tensors' device to the C ABI in include/ac.h, which documents the operators;
all arithmetic runs in libac's kernels.  Tensors are [B, H, L, d] in any strides
(d contiguous).  Nothing here synchronises but ops_status.

Gradients are calls of their own (rope_axes(inverse=True), window_attn_backward),
and rope_axes and window_attn make them where autograd records: for tensors that
require gradients, with new outputs.  window_attn has no second derivative and none
of its lse.  What is not recorded (outputs written into given tensors, the cache,
window_attn_backward itself) warns when one of its inputs requires gradients.

The common case of a call (new outputs, tensors on the current device) goes
through the compiled _fast module, which makes the same C calls; what it does
not take comes back as None and is checked, explained or done here.
"""
from __future__ import annotations

import ctypes
import functools
import importlib
import numbers
import operator
import os
import warnings
from typing import NamedTuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import ACCache8, ACView, ACWindow, check
from .build import FAST


def _load_fast():
    """The compiled module, or None: every call then takes the way through ctypes."""
    try:
        return importlib.import_module("._fast", __package__)
    except ImportError as e:
        if os.path.exists(FAST):
            warnings.warn(f"{FAST} does not load, calls go through ctypes (build again?): {e}", RuntimeWarning)
        return None


_fast = _load_fast()

_ROPE_DTYPES = {torch.bfloat16: _lib.AC_DTYPE_BF16, torch.float16: _lib.AC_DTYPE_F16, torch.float32: _lib.AC_DTYPE_F32}
_NO_VIEW = ACView(None, 0, 0, 0)


def _took(result):
    """Whether _fast made the call; raises what the library refused."""
    if result.__class__ is int:
        check(result)
    return result is not None


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, fn, *args):
    """fn(*args, stream) with `device` current."""
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if device.index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device.index))
    if status:
        check(status)


# ---------------------------------------------------------------- autograd
def _recorded(*tensors):
    """Whether autograd records what is done with one of them: backwards, or its tangent forwards."""
    tensors = [t for t in tensors if t is not None]
    return torch.is_grad_enabled() and any(t.requires_grad for t in tensors) or \
        getattr(forward_ad, "_current_level", -1) >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _warn_if_recorded(what, *tensors):
    if _recorded(*tensors):
        warnings.warn(f"{what} is not recorded by autograd: its result carries no gradients", UserWarning, stacklevel=3)


def _rows16(t):
    """t in strides that the attention takes (gradients come in any: broadcast, transposed)."""
    fits = t.data_ptr() % 16 == 0 and t.stride(3) == 1 and \
        all(n <= 1 or s > 0 and s % 8 == 0 for n, s in zip(t.shape[:3], t.stride()[:3]))
    return t if fits else t.clone(memory_format=torch.contiguous_format)


class _RopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inverse, args):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.inverse, ctx.args = inverse, args
        return _rope_now(q, k, positions, *args, inverse)

    @staticmethod
    def backward(ctx, gq, gk=None):
        positions, = ctx.saved_tensors
        grads = [g if n else None for g, n in zip((gq, gk), ctx.needs_input_grad)]
        given = [g if g.stride(3) == 1 else g.contiguous() for g in grads if g is not None]
        if not given:
            return None, None, None, None, None
        if _recorded(*given):  # (a rotation too)
            r = _RopeAxes.apply(given[0], given[1] if len(given) > 1 else None, positions, not ctx.inverse, ctx.args)
        else:
            r = _rope_now(given[0], given[1] if len(given) > 1 else None, positions, *ctx.args, not ctx.inverse)
        r = list(r) if len(given) > 1 else [r]
        return *(None if g is None else r.pop(0) for g in grads), None, None, None


class _WindowAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_lens, k_lens, rule, return_lse):
        ctx.set_materialize_grads(False)
        o, lse = _window_now(q, k, v, *rule, q_lens, k_lens, True)
        ctx.save_for_backward(q, k, v, o, lse, q_lens, k_lens)
        ctx.rule = rule
        return (o, lse) if return_lse else o

    @staticmethod
    @once_differentiable
    def backward(ctx, g, g_lse=None):
        if g_lse is not None:
            raise RuntimeError("window_attn: lse has no gradient")
        if g is None:
            return (None,) * 7
        q, k, v, o, lse, q_lens, k_lens = ctx.saved_tensors
        grads = _backward_now(_rows16(g), q, k, v, o, lse, *ctx.rule, q_lens, k_lens)
        return *(x if n else None for x, n in zip(grads, ctx.needs_input_grad)), None, None, None, None


def _shape(t, name):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, L, d], got {tuple(t.shape)}")
    return t.shape


def _view(t, name, device, shape, dtype=torch.bfloat16):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be [B, H, L, d] = {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    b, h, row, e = t.stride()
    if e != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return ACView(t.data_ptr(), b, h, row)


def _ints(t, name, device, shape):
    """Pointer of a contiguous int32 tensor, or None."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}")
    return t.data_ptr()


# ---------------------------------------------------------------- rotary embedding
def _arrays(freq, pairs):
    f, n = (ctypes.c_double * max(1, len(freq)))(*freq), (ctypes.c_int32 * max(1, len(pairs)))(*pairs)
    return f, n, ctypes.addressof(f), ctypes.addressof(n)


def _only(kind, *values):
    """Remembered by value are numbers alone (a tensor would be remembered as an object)."""
    if not all(isinstance(x, kind) for x in values):
        raise TypeError(f"{kind.__name__} numbers expected")


@functools.lru_cache(maxsize=64)
def _axes(pairs, theta):
    """Frequencies of the pairs: axis i has the series theta^(-k / pairs[i]) of its own."""
    _only(numbers.Integral, *pairs)
    _only(numbers.Real, *(theta if isinstance(theta, tuple) else (theta,)))
    theta = (theta,) * len(pairs) if not isinstance(theta, tuple) else theta
    if len(theta) != len(pairs) or any(n < 0 for n in pairs) or any(not t > 0 for t in theta):
        raise ValueError("one theta > 0 for all axes, or one for each; pairs >= 0")
    freq = [t ** (-k / n) for n, t in zip(pairs, theta) for k in range(n)]
    return _arrays(freq, pairs)


@functools.lru_cache(maxsize=64)
def _axes_given(pairs, freqs):
    _only(numbers.Integral, *pairs)
    _only(numbers.Real, *freqs)
    if len(freqs) != sum(pairs):
        raise ValueError("one frequency for each pair")
    return _arrays(freqs, pairs)


def rope_axes(q, k, positions, pairs, theta=10000.0, *, freqs=None, interleaved: bool = True, inverse: bool = False,
              out=None):
    """Rotate q [B, Hq, L, d] and k [B, Hk, L, d] (k may be None) by their tokens'
    positions along several axes (ac_rope_axes).

    positions: int32 [L, axes] or [B, L, axes]; pairs: how many of the d / 2
    element pairs turn with each axis, in order (what is left stays as it is);
    theta: base of the frequencies, one or one for each axis, or freqs: radians
    per step of each pair.  interleaved: pairs (2p, 2p + 1), otherwise
    (p, P + p).  inverse=True rotates back: the gradient with respect to the
    input is rope_axes(grad, ..., inverse=True), which autograd calls for new
    outputs.  out: (q, k) to write into, the inputs themselves allowed;
    contiguous new tensors otherwise.  bf16, fp16 or fp32.  Returns (q, k)
    rotated, or q alone when k is None."""
    pairs = tuple(pairs)
    axes = len(pairs)
    try:
        if freqs is not None:
            freq, npairs, pf, pn = _axes_given(pairs, tuple(freqs))
        else:
            freq, npairs, pf, pn = _axes(pairs, tuple(theta) if isinstance(theta, (list, tuple)) else theta)
    except TypeError:  # not plain numbers
        pairs = tuple(map(operator.index, pairs))
        if freqs is not None:
            freq, npairs, pf, pn = _axes_given(pairs, tuple(map(float, freqs)))
        else:
            freq, npairs, pf, pn = _axes(pairs, tuple(map(float, theta)) if isinstance(theta, (list, tuple)) else float(theta))
    args = (npairs, pf, pn, axes, freq, 1 if interleaved else 0)
    inverse = 1 if inverse else 0
    if out is None:
        if _fast is not None:
            r = _fast.rope(q, k, positions, pf, pn, axes, len(freq), args[5], inverse)
            if _took(r):
                return r
        if _recorded(q, k):
            return _RopeAxes.apply(q, k, positions, inverse, args)
    else:
        _warn_if_recorded("rope_axes(out=...)", q, k)
    return _rope_ctypes(q, k, positions, *args, inverse, out)


def _rope_now(q, k, positions, npairs, pf, pn, axes, freq, interleaved, inverse):
    """New outputs, whatever autograd thinks of the inputs."""
    if _fast is not None:
        r = _fast.rope(q, k, positions, pf, pn, axes, len(freq), interleaved, 1 if inverse else 0)
        if _took(r):
            return r
    return _rope_ctypes(q, k, positions, npairs, pf, pn, axes, freq, interleaved, inverse, None)


def _rope_ctypes(q, k, positions, npairs, pf, pn, axes, freq, interleaved, inverse, out):
    dt = q.dtype
    dtype = _ROPE_DTYPES.get(dt)
    if dtype is None:
        raise TypeError("q must be bf16, fp16 or fp32")
    dev = q.device
    shape = _shape(q, "q")
    vq = _view(q, "q", dev, shape, dt)
    B, Hq, L, d = shape
    if positions.dim() == 3:
        pos, pos_b = _ints(positions, "positions", dev, (B, L, axes)), L * axes
    else:
        pos, pos_b = _ints(positions, "positions", dev, (L, axes)), 0
    oq, ok = (None, None) if out is None else out
    if oq is None:
        oq = q.new_empty(shape)
    vqo = _view(oq, "out[0]", dev, shape, dt)
    Hk, vk, vko = 0, _NO_VIEW, _NO_VIEW
    if k is not None:
        Hk = _shape(k, "k")[1]
        kshape = (B, Hk, L, d)
        vk = _view(k, "k", dev, kshape, dt)
        if ok is None:
            ok = q.new_empty(kshape)
        vko = _view(ok, "out[1]", dev, kshape, dt)
    _on(dev, _lib.load().ac_rope_axes, dtype, vq, vqo, Hq, vk, vko, Hk, B, L, d, pos, pos_b, freq, npairs, axes,
        interleaved, 1 if inverse else 0)
    return oq if k is None else (oq, ok)


# ---------------------------------------------------------------- window attention
def _rule(left, right, sinks, block, scale):
    """The window's numbers as what the C struct holds."""
    n = tuple(map(operator.index, (left, right, sinks, block)))
    if any(not -2 ** 31 <= x < 2 ** 31 for x in n):
        raise ValueError(f"left, right, sinks and block must be 32-bit integers, got {n}")
    return *n, float(scale)


@functools.lru_cache(maxsize=1024)
def _window(left, right, sinks, block, scale):
    return ACWindow(left, right, sinks, block, scale)


@functools.lru_cache(maxsize=1024)
def _window_plan(left, right, sinks, block, scale, *sizes):
    """The window and the bytes of workspace of window_attn at these sizes."""
    n = ctypes.c_int64(0)
    w = _window(left, right, sinks, block, scale)
    check(_lib.load().ac_window_attn_workspace(*sizes, w, ctypes.byref(n)))
    return w, n.value


def _workspace(nbytes, like):
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def window_attn(q, k, v, *, left: int = -1, right: int = 0, sinks: int = 0, block: int = 1, q_lens=None, k_lens=None,
                scale: float = 0.0, out=None, return_lse: bool = False):
    """Softmax attention of q [B, Hq, Lq, d] over k, v [B, Hk, Lk, d] (bf16) within a
    window of `left` blocks back and `right` ahead (-1: no bound), blocks of
    `block` tokens, plus the first `sinks` tokens (ac_window_attn; struct
    ac_window says exactly which keys a query sees).  q_lens, k_lens: int32 [B]
    lengths of a padded batch.  Returns o, or (o, lse) with lse [B, Hq, Lq] fp32.
    Gradients of o pass through a new output (window_attn_backward); lse has none."""
    scale = float(scale)
    if out is None:
        if _fast is not None:
            r = _fast.window(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, bool(return_lse))
            if _took(r):
                return r
        if _recorded(q, k, v):
            return _WindowAttn.apply(q, k, v, q_lens, k_lens, (left, right, sinks, block, scale), bool(return_lse))
    else:
        _warn_if_recorded("window_attn(out=...)", q, k, v)
    return _window_ctypes(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, return_lse, out)


def _window_now(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, return_lse):
    """New outputs, whatever autograd thinks of the inputs."""
    if _fast is not None:
        r = _fast.window(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, return_lse)
        if _took(r):
            return r
    return _window_ctypes(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, return_lse, None)


def _window_ctypes(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, return_lse, out):
    dev = q.device
    shape = _shape(q, "q")
    B, Hq, Lq, d = shape
    _, Hk, Lk, _ = _shape(k, "k")
    kshape = (B, Hk, Lk, d)
    vq, vk, vv = _view(q, "q", dev, shape), _view(k, "k", dev, kshape), _view(v, "v", dev, kshape)
    if out is None:
        out = q.new_empty(shape)
    vo = _view(out, "out", dev, shape)
    lse = q.new_empty((B, Hq, Lq), dtype=torch.float32) if return_lse else None
    w, n = _window_plan(*_rule(left, right, sinks, block, scale), B, Hq, Hk, Lq, Lk, d)
    ws = _workspace(n, q)
    _on(dev, _lib.load().ac_window_attn, vq, vk, vv, vo, _ptr(lse), B, Hq, Hk, Lq, Lk, d,
        _ints(q_lens, "q_lens", dev, (B,)), _ints(k_lens, "k_lens", dev, (B,)), w, _ptr(ws), n)
    return (out, lse) if return_lse else out


@functools.lru_cache(maxsize=1024)
def _backward_plan(left, right, sinks, block, scale, *sizes):
    """The window and the bytes of workspace of window_attn_backward at these sizes."""
    n = ctypes.c_int64(0)
    w = _window(left, right, sinks, block, scale)
    check(_lib.load().ac_window_attn_backward_workspace(*sizes, w, ctypes.byref(n)))
    return w, n.value


def window_attn_backward(d_out, q, k, v, o, lse, *, left: int = -1, right: int = 0, sinks: int = 0, block: int = 1,
                         q_lens=None, k_lens=None, scale: float = 0.0, out=None):
    """Gradients (dq, dk, dv) of window_attn with the same window and lengths, from
    d_out, the gradient of o, and the o and lse that it returned
    (ac_window_attn_backward).  out: (dq, dk, dv) to write into."""
    scale = float(scale)
    if _fast is not None and out is None:
        r = _fast.backward(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens)
        if _took(r):
            return r
    _warn_if_recorded("window_attn_backward", d_out, q, k, v, o, lse)
    return _backward_ctypes(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens, out)


def _backward_now(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens):
    """New outputs, whatever autograd thinks of the inputs."""
    if _fast is not None:
        r = _fast.backward(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens)
        if _took(r):
            return r
    return _backward_ctypes(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens, None)


def _backward_ctypes(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens, out):
    dev = q.device
    qs = _shape(q, "q")
    B, Hq, Lq, d = qs
    _, Hk, Lk, _ = _shape(k, "k")
    ks = (B, Hk, Lk, d)
    vq, vk, vv = _view(q, "q", dev, qs), _view(k, "k", dev, ks), _view(v, "v", dev, ks)
    vo, vg = _view(o, "o", dev, qs), _view(d_out, "d_out", dev, qs)
    if lse.dtype is not torch.float32 or lse.shape != (B, Hq, Lq) or not lse.is_contiguous() or lse.device != dev:
        raise ValueError(f"lse must be a contiguous fp32 tensor {(B, Hq, Lq)} on {dev}")
    dq, dk, dv = (q.new_empty(qs), q.new_empty(ks), q.new_empty(ks)) if out is None else out
    w, n = _backward_plan(*_rule(left, right, sinks, block, scale), B, Hq, Hk, Lq, Lk, d)
    ws = _workspace(n, q)
    _on(dev, _lib.load().ac_window_attn_backward, vg, vq, vk, vv, vo, lse.data_ptr(), _view(dq, "dq", dev, qs),
        _view(dk, "dk", dev, ks), _view(dv, "dv", dev, ks), B, Hq, Hk, Lq, Lk, d,
        _ints(q_lens, "q_lens", dev, (B,)), _ints(k_lens, "k_lens", dev, (B,)), w, _ptr(ws), n)
    return dq, dk, dv


# ---------------------------------------------------------------- 8-bit cache
class Cache8(NamedTuple):
    """The tensors of a paged 8-bit cache: k, v float8_e4m3fn [pages, heads, page_tokens, d]
    and k_scale, v_scale fp32 [pages, heads], powers of two (struct ac_cache8)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, pages: int, heads: int, page_tokens: int, d: int, device="cuda"):
        """A cache that holds zeros."""
        k, v = (torch.zeros((pages, heads, page_tokens, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.full((pages, heads), 2.0 ** -120, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _cache(c, dev):
    k, v, ks, vs = c
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("cache.k must be [pages, heads, page_tokens, d]")
    pages, heads, T, d = shape
    for t in (k, v):
        if t.dtype is not torch.float8_e4m3fn or t.shape != shape or not t.is_contiguous() or t.device != dev:
            raise ValueError("cache.k and cache.v must be contiguous float8_e4m3fn tensors [pages, heads, page_tokens, d] "
                             f"on {dev}")
    for t in (ks, vs):
        if t.dtype is not torch.float32 or t.shape != (pages, heads) or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"cache.k_scale and cache.v_scale must be contiguous fp32 tensors [pages, heads] on {dev}")
    return ACCache8(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, heads, T, d)


def cache8_append(k, v, cache: Cache8, page_table, start, counts=None):
    """Write the new tokens k, v [B, heads, n, d] (bf16) of each sequence behind its
    first start[b] tokens into the cache (ac_cache8_append).  page_table: int32
    [B, max_pages]; start, counts: int32 [B] (counts: how many of the n are real)."""
    if _fast is not None and _took(_fast.append(k, v, *cache, page_table, start, counts)):
        return
    _warn_if_recorded("cache8_append", k, v)
    dev = k.device
    shape = _shape(k, "k")
    B, H, n, d = shape
    vk, vv = _view(k, "k", dev, shape), _view(v, "v", dev, shape)
    c = _cache(cache, dev)
    if H != c.heads or d != c.d:
        raise ValueError(f"k has {H} heads of {d}, the cache {c.heads} of {c.d}")
    if start is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages] and start [B]")
    per = page_table.shape[1]
    _on(dev, _lib.load().ac_cache8_append, c, vk, vv, B, n, _ints(page_table, "page_table", dev, (B, per)), per,
        _ints(start, "start", dev, (B,)), _ints(counts, "counts", dev, (B,)))


@functools.lru_cache(maxsize=1024)
def _cache_plan(left, right, sinks, block, scale, B, Hq, Lq, per, heads, T, d):
    """The window and the bytes of workspace of cache8_attn at these sizes."""
    n = ctypes.c_int64(0)
    w = _window(left, right, sinks, block, scale)
    sizes = ACCache8(256, 256, 256, 256, 0, heads, T, d)  # (addresses that are never read)
    check(_lib.load().ac_cache8_attn_workspace(sizes, B, Hq, Lq, per, w, ctypes.byref(n)))
    return w, n.value


def cache8_attn(q, cache: Cache8, page_table, k_lens, *, left: int = -1, right: int = 0, sinks: int = 0, block: int = 1,
                q_lens=None, scale: float = 0.0, out=None, return_lse: bool = False):
    """window_attn of q [B, Hq, Lq, d] over the first k_lens[b] cached tokens of each
    sequence (ac_cache8_attn)."""
    if _fast is not None and out is None:
        r = _fast.cache_attn(q, *cache, page_table, k_lens, left, right, sinks, block, float(scale), q_lens, bool(return_lse))
        if _took(r):
            return r
    _warn_if_recorded("cache8_attn", q)
    dev = q.device
    shape = _shape(q, "q")
    vq = _view(q, "q", dev, shape)
    B, Hq, Lq, d = shape
    c = _cache(cache, dev)
    if d != c.d:
        raise ValueError(f"q has heads of {d}, the cache of {c.d}")
    if k_lens is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages] and k_lens [B]")
    if out is None:
        out = q.new_empty(shape)
    vo = _view(out, "out", dev, shape)
    lse = q.new_empty((B, Hq, Lq), dtype=torch.float32) if return_lse else None
    per = page_table.shape[1]
    w, n = _cache_plan(*_rule(left, right, sinks, block, scale), B, Hq, Lq, per, c.heads, c.page_tokens, d)
    ws = _workspace(n, q)
    _on(dev, _lib.load().ac_cache8_attn, c, vq, vo, _ptr(lse), B, Hq, Lq, _ints(page_table, "page_table", dev, (B, per)), per,
        _ints(q_lens, "q_lens", dev, (B,)), _ints(k_lens, "k_lens", dev, (B,)), w, _ptr(ws), n)
    return (out, lse) if return_lse else out


def ops_status(device=None):
    """Wait for the current stream of `device` and raise ACError for what kernels of
    these operators have noted there since the last call: a length or page index
    out of range (AC_ERR_BOUNDS) or an expired wait (AC_ERR_TIMEOUT)."""
    _on(_cuda_device(device), _lib.load().ac_ops_status)


def ops_check_wait_timeout(limit_us: int, device=None):
    """Enqueue the bounded-wait health check of these operators
    (ac_ops_check_wait_timeout); the next ops_status raises with AC_ERR_TIMEOUT."""
    dev, fn = _cuda_device(device), _lib.load().ac_ops_check_wait_timeout
    _on(dev, functools.partial(fn, int(limit_us)))


def _cuda_device(device):
    dev = torch.device("cuda" if device is None else device)
    return torch.device("cuda", torch.cuda.current_device()) if dev.type == "cuda" and dev.index is None else dev
