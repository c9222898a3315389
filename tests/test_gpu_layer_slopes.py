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


def test_slopes_far_from_zero(Z):
    """The smooth activations' slopes at far pre-activations, relative to the slope itself.
    SiLU's is s (1 + h (1 - s)), s = 1 / (1 + e^-h): the argument of the hardware's exp2 is
    off by 2 half steps (its constant's rounding and the product's), which is 2 |h| 2^-24 of
    the power, exp2, sum and reciprocal by an ulp each and the polynomial by three half
    steps: (2 |h| + 12) 2^-24 of the slope down to h = -87, where s leaves the normal
    numbers; there the slope is below 88 * 2^-125. GELU's is far below any number at -32 (e
    to the -2390) and below e^-100 from -11 on."""
    z = torch.cat([torch.arange(-87.0, -15.0, 0.25), torch.tensor([-88.0, -89.0, -100.0, -127.0, -130.0, -1e3, -3e38,
                   float("-inf")]), torch.arange(20.0, 140.0), torch.tensor([1e3, 3e38, float("inf")])]).to(BF)
    say("slopes far from zero", z.numel())
    z = torch.unique(z)[None].to(dev())
    z64 = z.cpu().double().numpy()
    one = torch.ones(z.shape, dtype=F32, device=dev())
    got = Z.zero_dropout_grad(one, None, act=3, preact=z, dtype=F32).cpu().double().numpy()
    h = np.clip(z64, -700, 700)
    s = 1 / (1 + np.exp(-h))
    want = s * (1 + h * (1 - s))
    err = (2 * np.abs(h) + 12) * 2.0 ** -24 * np.abs(want)
    err = np.where(z64 < -87, 88 * 2.0 ** -125, err)
    bad = np.abs(got - want) > err
    assert not bool(bad.any()), (z64[bad][:8], got[bad][:8])
    got = Z.zero_dropout_grad(one, None, act=2, preact=z, dtype=F32).cpu().double().numpy()
    assert bool((got[z64 > 0] == 1).all()) and bool((np.abs(got[z64 < 0]) < np.exp(-100)).all())
