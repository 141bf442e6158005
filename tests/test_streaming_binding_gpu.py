"""The calls through ctypes do what those through the compiled module do, bit for bit."""
import pytest
import torch

from cluster_routed_sparse_b200 import streaming
from test_streaming_gpu import all_ops

pytestmark = pytest.mark.gpu


def test_both_ways_are_the_same(monkeypatch):
    assert streaming._fast is not None
    want = all_ops(11)()
    monkeypatch.setattr(streaming, "_fast", None)
    for a, b in zip(all_ops(11)(), want):
        assert torch.equal(a, b)
    streaming.ops_status()
