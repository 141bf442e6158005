"""A layer's exported state and its views are the same whatever lay in the memory that the context got: rows behind
the last cluster too."""
import numpy as np
import pytest
import torch

from _gpu_common import dev, gpu_state
from cluster_routed_sparse_b200 import synth
from cluster_routed_sparse_b200.api import SparseLayer

pytestmark = pytest.mark.gpu

CFG = synth.LayerConfig("state-L4096-H2-d64", 1, 2, 4096, 64, Cq=16, m0=32, n_max=128, tau_mode=synth.TAU_MEAN_FACTOR,
                        tau_value=1.0, topk=8, key_components=24)


def layer(cfg, n_max):
    return SparseLayer(1, cfg.H, cfg.L, cfg.d, Cq=cfg.Cq, m0=cfg.m0, n_max=n_max, tau_mode=cfg.tau_mode,
                       tau_value=cfg.tau_value, topk=cfg.topk, iters_q=cfg.iters_q, iters_k=cfg.iters_k, seed=5)


def test_state_does_not_depend_on_the_memory_before():
    Q, K, V = (dev(x) for x in synth.make_layer(CFG))
    blobs, states = [], []
    for n in range(4):
        # contexts of other layers leave their centres and selections behind, and one of them stays, so that the
        # driver keeps what the others had
        before = [layer(CFG, CFG.n_max + 8 * m) for m in range(2 * n)]
        for lay in before:
            lay.forward(Q, torch.randn_like(K) * (n + 1), V)
            lay.synchronize()
        for lay in before[::2]:
            lay.close()
        lay = layer(CFG, CFG.n_max)
        lay.forward(Q, K, V)
        lay.synchronize()
        blobs.append(lay.export_state())
        states.append(gpu_state(lay))
        for other in (lay, *before):
            other.close()
    assert all(b == blobs[0] for b in blobs)
    for s in states[1:]:
        for key in ("cent_k", "counts_k", "kmax", "kmin", "sel"):
            np.testing.assert_array_equal(s[key], states[0][key], err_msg=key)
