"""Out of memory is torch's own error, which programs catch to make room and go on."""
import pytest
import torch

import cluster_routed_sparse_b200 as crs

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs():
    x = torch.zeros(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    L = 2_000_000
    q, k = x.expand(1, 2000, L, 64), torch.zeros(1, 2000, 4, 64, device="cuda", dtype=torch.bfloat16)  # 512 GB, none of them held
    pos = torch.zeros(L, 1, device="cuda", dtype=torch.int32)
    with pytest.raises(torch.OutOfMemoryError):
        crs.rope_axes(q, None, pos, (32,))
    with pytest.raises(torch.OutOfMemoryError):
        crs.window_attn(q, k, k)
    y = crs.rope_axes(k, None, pos[:4], (32,))
    assert not y.any()
    crs.ops_status()
