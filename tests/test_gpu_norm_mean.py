"""GPU tests of a norm's mean: rows of one value, means that are large beside the differences,
and rows whose first element stands far out."""
import numpy as np
import pytest
import torch

import norm_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# one wave, four, eight of them to a row, one to four chunks a lane, odd ends, and rows read again
WIDTHS = [1, 7, 40, 513, 1001, 1500, 3001, 5000, 9001, 13001, 16001, 20011]


@pytest.mark.parametrize("N", WIDTHS)
def test_rows_of_one_value(Z, N):
    """Their differences are 0 and their mean is the value, however sums of it would round: y is the
    bias to the bit, 1 / sigma that of eps; with eps 0 it is infinite and y NaN."""
    values = torch.tensor([0.1, 10.3, 1000.1, -7.7e-5, 123456.7, 3e30, 0.0, 65504.0], device=dev())
    g = torch.Generator(device=dev()).manual_seed(N)
    w, b = (torch.randn(N, generator=g, device=dev()).to(BF) for _ in range(2))
    x = values[:, None].expand(-1, N).contiguous()
    say("rows of one value", N)
    want = 1.0 / np.sqrt(np.float32(1e-5))
    for xt, kw in ((x, {}), (x.to(BF), {}), (0.25 * x, dict(residual=0.75 * x)),
                   (x.to(BF), dict(residual=x.to(BF) * 2))):
        got = Z.zero_norm_forward(xt, w, b, stats=True, dtype=F32, **kw)
        y, s, stats = got if kw else (got[0], xt, got[1])
        assert torch.equal(y, b.float()[None].expand_as(y))
        assert torch.equal(stats[:, 0], s[:, 0].float())
        assert float((stats[:, 1] / float(want) - 1).abs().max()) <= 3 * 2.0 ** -24
        y, *_, stats = Z.zero_norm_forward(xt, w, b, stats=True, dtype=F32, eps=0.0, **kw)
        assert bool(y.isnan().all()) and bool(stats[:, 1].isinf().all())


@pytest.mark.parametrize("N", [700, 1001, 4001, 12000, 20011])
@pytest.mark.parametrize("mean,sigma", [(1000.0, 0.01), (-30.0, 1e-3), (1.0, 1e-5)])
def test_a_mean_that_is_large_beside_the_differences(Z, N, mean, sigma):
    """The mean m is within half of it or twice it of every element, so that the differences are exact,
    and what they have left of the mean is summed on its own: that sum, the variance's and the
    few operations behind them leave (depth + 8) u each of y and of 1, twice that together, to first
    order; another factor of two covers the variance's own difference to the mean of the squares,
    as m is off by a step of 32 bits at most and sigma is 80 of them or more."""
    rng = np.random.default_rng(N)
    x = (mean + sigma * rng.standard_normal((4, N))).astype(np.float32)
    say("large mean", N, mean, sigma)
    y, stats = Z.zero_norm_forward(torch.from_numpy(x).to(dev()), eps=0.0, stats=True, dtype=F32)
    x = x.astype(np.float64)
    m = x.mean(1, keepdims=True)
    want = (x - m) / np.sqrt(((x - m) ** 2).mean(1, keepdims=True))
    off = np.abs(y.cpu().double().numpy() - want)
    assert (off <= 4 * (R.depth(N) + 8) * R.u * (1 + np.abs(want))).all(), float(off.max())
    # the mean is one rounding of 32 bits away
    assert np.abs(stats[:, 0].cpu().double().numpy() - m[:, 0]).max() <= 2.0 ** -24 * 1.01 * abs(mean)


@pytest.mark.parametrize("N", [40, 1001, 3001, 9001, 20011])
def test_a_first_element_far_from_the_others(Z, N):
    """The differences to it round as it does; the mean does not depend on them."""
    rng = np.random.default_rng(N)
    x = rng.standard_normal((6, N)).astype(np.float32)
    x[:, 0] = [30.0, -300.0, 3e3, 3e4, -3e5, 3e6]
    say("far first element", N)
    y, stats = Z.zero_norm_forward(torch.from_numpy(x).to(dev()), stats=True, dtype=F32)
    want, err, st, es = R.forward(x.astype(np.float64), np.ones(N), np.zeros(N), rms=False, eps=1e-5, out="f32")
    assert (np.abs(y.cpu().double().numpy() - want) <= err).all()
    assert (np.abs(stats.cpu().double().numpy() - st) <= es + 2.0 ** -140).all()


@pytest.mark.parametrize("over", ["x", "residual"])
def test_long_rows_in_place(Z, over):
    """The row's first element is taken before anything is written over it."""
    g = torch.Generator(device=dev()).manual_seed(5)
    x, r = (torch.randn(300, 20011, generator=g, device=dev()) + 50 for _ in range(2))
    want = Z.zero_norm_forward(x, residual=r, stats=True)
    a, b = x.clone(), r.clone()
    got = Z.zero_norm_forward(a, residual=b, sum=a if over == "x" else b, stats=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("N", [40, 3001, 20011])
def test_infinities_by_the_formula(Z, N):
    """Layer: the mean is infinite and all differences, and y, NaN. RMS: 1 / sigma is 0, the
    infinity's own place 0 times infinity, the others the bias."""
    g = torch.Generator(device=dev()).manual_seed(N)
    x = torch.randn(4, N, generator=g, device=dev())
    b = torch.randn(N, generator=g, device=dev()).to(BF)
    x[1, N // 3], x[2, 5], x[3, 2] = float("inf"), float("-inf"), float("nan")
    for xt in (x, x.to(BF)):
        y = Z.zero_norm_forward(xt, None, b, dtype=F32)
        assert bool(y[1:].isnan().all()) and bool(y[0].isfinite().all())
        y, stats = Z.zero_norm_forward(xt, None, b, kind=Z.ZERO_NORM_RMS, stats=True, dtype=F32)
        for row, at in ((1, N // 3), (2, 5)):
            others = torch.arange(N, device=dev()) != at
            assert bool(y[row, at].isnan()) and torch.equal(y[row][others], b.float()[others])
            assert float(stats[row, 1]) == 0.0 and float(stats[row, 0]) == 0.0
        assert bool(y[3].isnan().all()) and bool(y[0].isfinite().all())
    # squares beyond fp32
    y = Z.zero_norm_forward(torch.full((2, N), 1e30, device=dev()), None, b, kind=Z.ZERO_NORM_RMS, dtype=F32)
    assert torch.equal(y, b.float()[None].expand_as(y))
    for eps in (-1e-9, 2e30, float("inf"), float("nan")):
        with pytest.raises(Z.ZeroError, match="eps"):
            Z.zero_norm_forward(x, eps=eps)
