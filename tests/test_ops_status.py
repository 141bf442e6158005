"""Arguments that the health check of the streaming operators refuses, without a GPU."""
import pytest

import cluster_routed_sparse_b200 as crs
from cluster_routed_sparse_b200 import _lib


@pytest.mark.parametrize("limit", [0, -5, 2000001])
def test_wait_limits_out_of_range(limit):
    assert _lib.load().ac_ops_check_wait_timeout(limit, None) == _lib.AC_ERR_INVALID_ARG


def test_only_on_a_gpu():
    with pytest.raises(ValueError):
        crs.ops_check_wait_timeout(1000, "cpu")
