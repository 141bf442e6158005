"""What kernels of the streaming operators note on the device reaches ops_status: expired waits and bad pages,
each once, whatever else is noted and asked for at the same time."""
import time

import pytest
import torch

import cluster_routed_sparse_b200 as crs
from cluster_routed_sparse_b200 import _lib
from test_streaming_gpu import gen, normal

pytestmark = pytest.mark.gpu


def status():
    try:
        crs.ops_status()
    except _lib.ACError as e:
        return e.status
    return _lib.AC_OK


def test_an_expired_wait_is_reported_once():
    """A wait for something that nothing does ends after its limit, and calls after it work."""
    q, k, v = (normal(gen(n), 1, 2, 300, 64) for n in range(3))
    want = crs.window_attn(q, k, v, return_lse=True)
    grads = crs.window_attn_backward(q, q, k, v, *want)
    assert status() == _lib.AC_OK
    t0 = time.perf_counter()
    crs.ops_check_wait_timeout(20000)
    assert status() == _lib.AC_ERR_TIMEOUT
    assert 0.019 <= time.perf_counter() - t0 < 1.5
    assert status() == _lib.AC_OK
    for a, b in zip(want + grads, crs.window_attn(q, k, v, return_lse=True) + crs.window_attn_backward(q, q, k, v, *want)):
        assert torch.equal(a, b)
    assert status() == _lib.AC_OK
    crs.ops_check_wait_timeout(1000)  # noted, not yet asked for: later launches do their work all the same
    again = crs.window_attn(q, k, v)
    assert status() == _lib.AC_ERR_TIMEOUT and torch.equal(again, want[0])


def test_a_note_made_while_another_is_reported_is_kept():
    """A bad page on one stream, again and again, while expired waits on another are noted and reported: the
    report of the one never takes the other along."""
    c = crs.Cache8.empty(2, 1, 16, 64)
    k = normal(gen(1), 1, 1, 1, 64)
    table = torch.full((1, 1), 9, device="cuda", dtype=torch.int32)
    start = torch.zeros(1, device="cuda", dtype=torch.int32)
    crs.cache8_append(k, k, c, table, start)
    assert status() == _lib.AC_ERR_BOUNDS and status() == _lib.AC_OK
    pages, waits = torch.cuda.Stream(), torch.cuda.Stream()
    expired = 0
    for n in range(300):
        with torch.cuda.stream(waits):
            crs.ops_check_wait_timeout(1)
        spin = n * 7 % 300  # the other note comes at another moment of the report each time
        with torch.cuda.stream(pages):
            torch.cuda._sleep(spin * 100)
            crs.cache8_append(k, k, c, table, start)
        with torch.cuda.stream(waits):
            seen = [status()]
        torch.cuda.synchronize()
        for _ in range(2):
            seen.append(status())
        assert sorted(seen) == [_lib.AC_OK, _lib.AC_ERR_TIMEOUT, _lib.AC_ERR_BOUNDS], (n, seen)
        expired += seen[0] == _lib.AC_ERR_TIMEOUT
    assert expired
