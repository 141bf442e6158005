"""What the streaming operators refuse, through the C ABI and through the binding,
without a GPU: every call here has an argument that is refused before any device
work."""
import ctypes

import pytest
import torch

import cluster_routed_sparse_b200 as crs
from cluster_routed_sparse_b200 import _lib
from cluster_routed_sparse_b200._lib import (AC_ERR_INVALID_ARG as INVALID, AC_ERR_UNSUPPORTED as UNSUPPORTED,
                                             AC_ERR_WORKSPACE as WORKSPACE, ACCache8, ACView, ACWindow)

A = 1 << 20  # an aligned address that is never read


def view(p=A, b=1 << 16, h=1 << 12, l=64):
    return ACView(p, b, h, l)


def window(left=3, right=0, sinks=0, block=1, scale=0.0):
    return ACWindow(left, right, sinks, block, scale)


def rope(dtype=0, x=view(), y=view(), H=2, B=1, L=4, d=64, pos=A, freq=(1.0,) * 32, pairs=(32,), n_axes=1):
    f, p = (ctypes.c_double * len(freq))(*freq), (ctypes.c_int32 * len(pairs))(*pairs)
    return _lib.load().ac_rope_axes(dtype, x, y, H, None, None, 0, B, L, d, pos, 0, f, p, n_axes, 1, 0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(d=63), UNSUPPORTED), (dict(d=258), UNSUPPORTED),
    (dict(pairs=(33,), freq=(1.0,) * 33), INVALID), (dict(pairs=(-1,)), INVALID), (dict(n_axes=0), INVALID),
    (dict(freq=(float("nan"),) * 32), INVALID), (dict(x=None), INVALID), (dict(y=view(p=None)), INVALID),
    (dict(y=view(h=0)), INVALID), (dict(y=view(l=0)), INVALID), (dict(B=2, y=view(b=0)), INVALID),
    (dict(pos=None), INVALID), (dict(B=-1), INVALID), (dict(H=70000), INVALID),
])
def test_rope_refusals(kw, expect):
    assert rope(**kw) == expect
    assert _lib.load().ac_last_error_string(None)


def attn(q=view(), k=view(), v=view(), o=view(), B=1, Hq=4, Hk=2, Lq=8, Lk=8, d=64, w=window(), ws=A, nbytes=1 << 40):
    return _lib.load().ac_window_attn(q, k, v, o, None, B, Hq, Hk, Lq, Lk, d, None, None, w, ws, nbytes, None)


def backward(q=view(), k=view(), v=view(), o=view(), B=1, Hq=4, Hk=2, Lq=8, Lk=8, d=64, w=window(), ws=A,
             nbytes=1 << 40, lse=A):
    return _lib.load().ac_window_attn_backward(o, q, k, v, o, lse, q, k, v, B, Hq, Hk, Lq, Lk, d, None, None, w, ws,
                                               nbytes, None)


BAD_SIZES = [
    (dict(d=96), UNSUPPORTED), (dict(Hk=3), INVALID), (dict(Hk=0), INVALID), (dict(Hq=300, Hk=2), INVALID),
    (dict(B=-1), INVALID), (dict(Lq=-1), INVALID), (dict(Lk=(1 << 30) + 1), INVALID), (dict(B=70000), INVALID),
    (dict(B=1000, Hq=1000, Hk=1000, Lq=1 << 20, Lk=1), INVALID),
    (dict(w=window(left=-2)), INVALID), (dict(w=window(right=-2)), INVALID), (dict(w=window(sinks=-1)), INVALID),
    (dict(w=window(block=0)), INVALID), (dict(w=window(scale=float("inf"))), INVALID), (dict(w=None), INVALID),
    (dict(w=window(scale=-0.1)), INVALID), (dict(q=None), INVALID), (dict(q=view(p=None)), INVALID), (dict(k=view(p=A + 8)), INVALID),
    (dict(v=view(l=63)), INVALID), (dict(k=view(h=0)), INVALID), (dict(q=view(l=-64)), INVALID),
    (dict(o=view(h=4)), INVALID),
]


@pytest.mark.parametrize("kw,expect", BAD_SIZES)
@pytest.mark.parametrize("fn", [attn, backward])
def test_window_attn_refusals(fn, kw, expect):
    assert fn(**kw) == expect


def test_workspaces_are_checked():
    lib = _lib.load()
    n = ctypes.c_int64(-1)
    assert lib.ac_window_attn_workspace(1, 4, 2, 1, 1 << 20, 64, window(-1), ctypes.byref(n)) == 0
    if n.value:
        assert attn(Lq=1, Lk=1 << 20, w=window(-1), nbytes=n.value - 1) == WORKSPACE
        assert attn(Lq=1, Lk=1 << 20, w=window(-1), ws=None, nbytes=n.value) == WORKSPACE
    assert lib.ac_window_attn_backward_workspace(1, 4, 2, 8, 8, 64, window(), ctypes.byref(n)) == 0
    if n.value:
        assert backward(nbytes=n.value - 1) == WORKSPACE
    assert lib.ac_window_attn_workspace(1, 4, 2, 8, 8, 64, window(), None) == INVALID
    assert lib.ac_window_attn_backward_workspace(1, 4, 2, 8, 8, 64, window(), None) == INVALID
    assert backward(lse=None) == INVALID


def cache(k=A, v=A, pages=4, heads=2, tokens=16, d=64):
    return ACCache8(k, v, A, A, pages, heads, tokens, d)


@pytest.mark.parametrize("c,expect", [
    (cache(d=96), UNSUPPORTED), (cache(tokens=48), UNSUPPORTED), (cache(tokens=0), UNSUPPORTED),
    (cache(k=None), INVALID), (cache(v=A + 4), INVALID), (cache(heads=0), INVALID), (cache(pages=-1), INVALID), (None, INVALID),
])
def test_cache_refusals(c, expect):
    lib = _lib.load()
    assert lib.ac_cache8_append(c, view(), view(), 1, 4, A, 2, A, None, None) == expect
    assert lib.ac_cache8_attn(c, view(), view(), None, 1, 4, 1, A, 2, None, A, window(), A, 1 << 40, None) == expect


def test_cache_call_refusals():
    lib, c = _lib.load(), cache()
    assert lib.ac_cache8_append(c, view(), view(), 1, 4, None, 2, A, None, None) == INVALID
    assert lib.ac_cache8_append(c, view(), view(), 1, 4, A, 2, None, None, None) == INVALID
    assert lib.ac_cache8_append(c, view(l=8 + 4), view(), 1, 4, A, 2, A, None, None) == INVALID
    assert lib.ac_cache8_append(c, view(), view(), -1, 4, A, 2, A, None, None) == INVALID
    assert lib.ac_cache8_append(c, view(), view(), 1, 4, A, -1, A, None, None) == INVALID
    for kw in (dict(Hq=3), dict(table=None), dict(lens=None), dict(w=window(sinks=-1)), dict(pages=1 << 27)):
        kw = {**dict(Hq=4, table=A, lens=A, w=window(), pages=2), **kw}
        assert lib.ac_cache8_attn(c, view(), view(), None, 1, kw["Hq"], 1, kw["table"], kw["pages"], None, kw["lens"],
                                  kw["w"], A, 1 << 40, None) == INVALID


def test_binding_refusals():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: crs.rope_axes(x, None, pos, (32,)),                       # not on a GPU
                 lambda: crs.rope_axes(x, x[:, :, :3], pos, (32,)),
                 lambda: crs.rope_axes(x, None, pos.long(), (32,)),
                 lambda: crs.rope_axes(x, None, pos, (16, 16)),
                 lambda: crs.rope_axes(x, None, pos, (32,), freqs=[1.0]),
                 lambda: crs.rope_axes(x, None, pos, (32,), theta=-1.0),
                 lambda: crs.rope_axes(x, None, pos, (16, 16), theta=(10.0,)),
                 lambda: crs.window_attn(x, x, x),
                 lambda: crs.window_attn(x, x, x[:, :1]),
                 lambda: crs.window_attn(x.transpose(2, 3), x, x),
                 lambda: crs.window_attn(x, x, x, q_lens=torch.zeros(2, dtype=torch.int32)),
                 lambda: crs.cache8_attn(x, crs.Cache8.empty(2, 2, 16, 128, "cpu"), pos, pos[0]),
                 lambda: crs.cache8_append(x, x, crs.Cache8.empty(2, 3, 16, 64, "cpu"), pos, pos[0]),
                 lambda: crs.ops_status("cpu")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: crs.rope_axes(x.double(), None, pos, (32,)), lambda: crs.window_attn(x.float(), x, x),
                 lambda: crs.rope_axes(x, x.float(), pos, (32,))):
        with pytest.raises(TypeError):
            call()


def test_workspaces_are_aligned():
    assert backward(ws=A + 16) == INVALID
    lib, n = _lib.load(), ctypes.c_int64(-1)
    assert lib.ac_window_attn_workspace(1, 4, 2, 1, 1 << 20, 64, window(-1), ctypes.byref(n)) == 0 and n.value
    assert attn(Lq=1, Lk=1 << 20, w=window(-1), ws=A + 128) == INVALID


@pytest.mark.parametrize("kw", [dict(left=2 ** 40), dict(left=2 ** 32 - 1), dict(right=2 ** 31), dict(sinks=2 ** 32 + 4),
                                dict(block=2 ** 32 + 1)])
def test_window_numbers_that_32_bits_do_not_hold(kw):
    """Not taken modulo 2^32, which would be another window."""
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    lse, ints = torch.zeros(1, 2, 4), torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: crs.window_attn(x, x, x, **kw), lambda: crs.window_attn_backward(x, x, x, x, x, lse, **kw),
                 lambda: crs.cache8_attn(x, crs.Cache8.empty(2, 2, 16, 64, "cpu"), ints, ints[0, :1], **kw)):
        with pytest.raises(ValueError, match="32-bit"):
            call()


def test_rope_numbers_are_read_by_value():
    """A tensor among them is read at the call, not remembered as an object."""
    from cluster_routed_sparse_b200 import streaming
    x, pos = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 1, dtype=torch.int32)
    theta, pairs = torch.tensor(100.0), torch.tensor([32])
    streaming._axes.cache_clear()
    for n in range(3):
        theta += 1
        for _ in range(2):
            with pytest.raises(ValueError, match="CUDA"):
                crs.rope_axes(x, None, pos, pairs, theta)
        assert streaming._axes.cache_info().currsize == n + 1
