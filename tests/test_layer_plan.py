"""Which calls split their reduction over workgroups, as the workspace shows it (CPU only)."""
import pytest

import zero_partitioned_optimizer_amd as Z


@pytest.mark.parametrize("rows,long,narrow", [(1, 50257, 64), (4, 16384, 16), (16, 8192, 128), (1, 16384, 768)])
def test_long_narrow_reductions_are_split(rows, long, narrow):
    """A handful of workgroups would stream the weights with most of the chip idle."""
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_FORWARD, Z.ZERO_W_OUT_IN, rows, long, narrow) > 0
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_GRAD_INPUT, Z.ZERO_W_IN_OUT, rows, narrow, long) > 0


@pytest.mark.parametrize("rows,K,N", [(1, 768, 2304), (4, 2040, 4096), (16, 768, 768), (1, 64, 50257)])
def test_short_reductions_are_not(rows, K, N):
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_FORWARD, Z.ZERO_W_OUT_IN, rows, K, N) == 0
