"""Which calls split their reduction over workgroups, as the workspace shows it (CPU only)."""
import pytest

import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import _binding as B, layer


@pytest.mark.parametrize("rows,long,narrow", [(1, 50257, 64), (4, 16384, 16), (16, 8192, 128), (1, 16384, 768)])
def test_long_narrow_reductions_are_split(rows, long, narrow):
    """A handful of workgroups would stream the weights with most of the chip idle."""
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_FORWARD, Z.ZERO_W_OUT_IN, rows, long, narrow) > 0
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_GRAD_INPUT, Z.ZERO_W_IN_OUT, rows, narrow, long) > 0


@pytest.mark.parametrize("rows,K,N", [(1, 768, 2304), (4, 2040, 4096), (16, 768, 768), (1, 64, 50257)])
def test_short_reductions_are_not(rows, K, N):
    assert Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_FORWARD, Z.ZERO_W_OUT_IN, rows, K, N) == 0


def test_split_rows_refuse_no_workspace():
    """Odd rows of a long reduction are split, with a workspace or not at all."""
    base = 1 << 40
    a = Z.zero_linear_args(M=1, K=4097, N=64, x=base, ld_x=4097, w=base + 0x10000, ld_w=4097, y=base + 0x200000, ld_y=64,
                           y_dtype=Z.ZERO_BF16)
    assert layer._lib().zero_linear_forward(a, None) == B.ZERO_E_INVAL and "workspace_dev" in Z.zero_last_error()
