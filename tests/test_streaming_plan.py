"""How the gradients of the window attention divide the work of key tiles that many queries see, read off the
workspace that they ask for (fp32 dK and dV of 128 keys for each part), without a GPU."""
import ctypes

import pytest

from cluster_routed_sparse_b200 import _lib


def parts_of(L, left, sinks, d=64):
    """Key tiles that may have parts, times the most parts of one: of one head with itself as keys."""
    n = ctypes.c_int64(0)
    w = _lib.ACWindow(left, 0, sinks, 1, 0.0)
    assert _lib.load().ac_window_attn_backward_workspace(1, 1, 1, L, L, d, w, ctypes.byref(n)) == 0
    stats = -(-L // 128) * 256 * 4
    assert (n.value - stats) % (2 * 128 * d * 4) == 0
    return (n.value - stats) // (2 * 128 * d * 4)


def test_first_tokens_do_not_count_among_the_queries_of_other_keys():
    # 64 tiles of first tokens that all 256 query tiles see, 192 others that 6 see: about 17,500 tile pairs for twice
    # 148 SMs, 59 to a part, 5 parts
    assert parts_of(32760, 511, 8192) == 64 * 5


@pytest.mark.parametrize("L,left,sinks", [(8192, 127, 2048), (8192, 63, 1024), (4096, 200, 2000)])
def test_only_first_tokens_come_in_parts(L, left, sinks):
    # the others have 2 to 5 query tiles, fewer than the eight that a part holds at least
    first, tiles = -(-sinks // 128), L // 128
    assert parts_of(L, left, sinks) == first * -(-tiles // 8)


def test_no_first_tokens_no_parts():
    assert parts_of(8192, 127, 0) == 0
