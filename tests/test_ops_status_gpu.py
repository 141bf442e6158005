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
