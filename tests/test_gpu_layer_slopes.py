"""Slopes of the activations at pre-activations of no ordinary size: NaN, and values so
negative that a slope is tiny, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("act", [1, 2, 3])
def test_slopes_of_nan(Z, act):
    """ReLU's slope is 1 where z > 0 and 0 elsewhere, at a NaN too; the smooth
    activations' slopes at a NaN are NaN, except behind a dropped element."""
    M, N = 70, 136
    rng = np.random.default_rng(31)
    say("slopes of nan", act)
    z = rng.standard_normal((M, N)).astype(np.float32)
    z[rng.random((M, N)) < 0.3] = np.nan
    z[11] = np.nan
    zt = torch.from_numpy(z).to(dev()).to(BF)
    z64 = zt.cpu().double().numpy()
    drop = Z.zero_dropout(0.25, 8, 9)
    keep = R.drop_factor(M, N, 0.25, 8, 9) != 0
    one = torch.ones((M, N), dtype=BF, device=dev())
    got = [(Z.zero_dropout_grad(one, None, act=act, preact=zt, dtype=F32), np.ones_like(keep)),
           (Z.zero_dropout_grad(one, drop, act=act, preact=zt, dtype=F32), keep)]
    eye = torch.eye(N, dtype=BF, device=dev())
    got += [(Z.zero_linear_grad_input(one, eye, act=act, preact=zt, dtype=F32), np.ones_like(keep)),
            (Z.zero_linear_grad_input(one[:3], eye, act=act, preact=zt[:3], dropout=drop, dtype=F32), keep[:3])]
    for g, k in got:
        g = g.cpu().double().numpy()
        s = R.slope(R.ACTS[act], z64[:len(g)])
        assert np.array_equal(np.isnan(g), np.isnan(s) & k)
        if act == 1:
            assert np.array_equal(g != 0, (s != 0) & k)
