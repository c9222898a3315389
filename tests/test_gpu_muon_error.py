"""GPU tests of how near the orthogonalisation is to its formula in 64 bits: nearer than o's
rounding lets one see directly, by what is left beyond half a step of each element
(tests/muon_error_ref.py says what arithmetic of 32 bits may leave)."""
import numpy as np
import pytest
import torch

import muon_error_ref as E
from gpu_util import dev, say

pytestmark = pytest.mark.gpu


def run(Z, x, **kw):
    return Z.zero_orthogonalize(torch.from_numpy(x).to(dev()), **kw).cpu().double().numpy()


@pytest.mark.parametrize("kind,rows,cols,steps", E.CASES)
def test_near_the_formula(Z, kind, rows, cols, steps):
    x = E.matrix(kind, rows, cols, np.random.default_rng(rows * 1000 + cols)).astype(np.float32)
    say("orthogonalize", kind, rows, cols, steps)
    E.check(run(Z, x, steps=steps)[None], x.astype(np.float64)[None], (kind, rows, cols, steps), steps=steps)


@pytest.mark.parametrize("shape", [(2, 200, 300), (2, 300, 200)], ids=str)
def test_a_table_of_larger_gains(Z, shape):
    rng = np.random.default_rng(4)
    x = np.stack([E.matrix(k, *shape[1:], rng) for k in ("rank6", "normal")]).astype(np.float32)
    say("orthogonalize with a table", shape)
    E.check(run(Z, x, coefficients=E.TABLE), x.astype(np.float64), shape, coefficients=E.TABLE)


@pytest.mark.parametrize("size", [(40, 256, 512), (12, 768, 2304), (1, 2304, 4096), (1, 4096, 1000)], ids=str)
def test_near_the_formula_by_every_kind_of_tile(Z, size):
    """A few strong directions over noise, as momenta are, the formula in 64 bits on the device."""
    B, r, c = size
    g = torch.Generator(device=dev()).manual_seed(r + c)
    x = torch.randn(B, r, 12, generator=g, device=dev()) @ torch.randn(B, 12, c, generator=g, device=dev())
    x += 0.3 * torch.randn(B, r, c, generator=g, device=dev())
    say("orthogonalize", size)
    o = Z.zero_orthogonalize(x)
    pick = sorted({0, B // 2, B - 1})
    X = x[pick].double().cpu().numpy()
    if r * c <= 768 * 2304:
        E.check(o[pick].double().cpu().numpy(), X, size)
        return
    # too large for the host: the same sums, the allowance with s = 1.3, above the largest
    # singular value of any iterate of the default coefficients
    X = x.double()
    X = X / X.square().sum((1, 2), keepdim=True).sqrt()
    X = X.transpose(1, 2).contiguous() if r > c else X
    a, b, c5 = E.R.COEF
    s = 1.3
    at = np.linspace(0, s, 200)
    gain = np.abs(a + 3 * b * at ** 2 + 5 * c5 * at ** 4).max()
    fresh = 2.0 ** -23 * (abs(a) + abs(b) * s ** 2 + abs(c5) * s ** 4)
    error = 2.0 ** -23
    for _ in range(5):
        error = error * gain + fresh * float(X.norm())
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.bmm(b * A + c5 * torch.bmm(A, A), X)
    want = (X.transpose(1, 2) if r > c else X).cpu().numpy()
    off = E.beyond_rounding(o.double().cpu().numpy(), want)
    assert off <= 2 * error, (off, 2 * error, float(X.norm()))


@pytest.mark.parametrize("tall", [False, True])
def test_what_passes_the_range_is_nan(Z, tall):
    """Elements of X from 16 and of A and b A + c A A from 64 on, in a middle step: NaN all over, in
    that matrix alone. An element (0, 1) of the last step's b A + c A A: rows (or columns) 0 and 1,
    and the others are the formula's, which does not use it for them."""
    rng = np.random.default_rng(9)

    def run_both(x, **kw):
        other = rng.standard_normal(x.shape).astype(np.float32)
        both = np.stack([x, other, x])
        o = run(Z, np.ascontiguousarray(both.transpose(0, 2, 1)) if tall else both, **kw)
        return o.transpose(0, 2, 1) if tall else o, other

    # rows 0 and 1 half alike, the others orthogonal to all: A is 0.1 at (0, 1) and 0.2 on the diagonal
    q = np.linalg.qr(rng.standard_normal((300, 5)))[0].T
    q[1] = 0.5 * q[0] + np.sqrt(0.75) * q[1]
    x = q.astype(np.float32)
    kw = dict(steps=1, coefficients=(1.0, 1000.0, 0.0))
    say("beyond the range", tall)
    o, _ = run_both(x, **kw)
    assert np.isnan(o[0, :2]).all() and np.isnan(o[2, :2]).all()
    want = E.R.orthogonalize(x, **kw)[2:]
    # 201 x, its roundings in 32 bits a hundredth of bf16's half step
    assert np.abs(o[[0, 2], 2:] - want).max() <= 2.0 ** -8 * np.abs(want).max() * 1.01
    # X of one large element: 0.9 * 20 in the second step
    x = np.full((5, 300), 0.01, np.float32)
    x[3, 7] = 1.0
    o, _ = run_both(x, steps=2, coefficients=[(20.0, 0.0, 0.0), (1.0, -0.5, 0.0)])
    assert np.isnan(o[[0, 2]]).all() and np.isfinite(o[1]).all()
    # A of rank 1, 8100 / 64 off its diagonal in the second step, X's own elements 90 / 140
    x = np.ones((64, 300), np.float32)
    o, _ = run_both(x, steps=2, coefficients=[(90.0, 0.0, 0.0), (1.0, -0.5, 0.0)])
    assert np.isnan(o[[0, 2]]).all()


@pytest.mark.parametrize("size", E.PLAN_SIZES, ids=str)
def test_near_the_formula_however_the_products_are_cut(Z, size):
    """Every kind of tile, whole, split in one part and in two, of wide and tall matrices, against the
    formula in 64 bits on the device, matrix by matrix; the allowance with s = 1.3 as above."""
    B, r, c = size
    g = torch.Generator(device=dev()).manual_seed(r * c)
    x = torch.randn(B, r, 12, generator=g, device=dev()) @ torch.randn(B, 12, c, generator=g, device=dev())
    x += 0.3 * torch.randn(B, r, c, generator=g, device=dev())
    say("orthogonalize", size)
    o = Z.zero_orthogonalize(x)
    assert torch.equal(o, Z.zero_orthogonalize(x))
    X = x.double()
    X = X / X.square().sum((1, 2), keepdim=True).sqrt()
    X = X.transpose(1, 2).contiguous() if r > c else X
    ca, cb, cc = E.R.COEF
    at = np.linspace(0, 1.3, 200)
    gain = np.abs(ca + 3 * cb * at ** 2 + 5 * cc * at ** 4).max()
    fresh = 2.0 ** -23 * (abs(ca) + abs(cb) * 1.3 ** 2 + abs(cc) * 1.3 ** 4)
    error = torch.full((B,), 2.0 ** -23, dtype=torch.float64, device=dev())
    for _ in range(5):
        error = error * gain + fresh * X.square().sum((1, 2)).sqrt()
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = ca * X + torch.bmm(cb * A + cc * torch.bmm(A, A), X)
    o = o.double()
    o = o.transpose(1, 2) if r > c else o
    half = torch.ldexp(torch.ones_like(X), torch.frexp(torch.maximum(o.abs(), X.abs())).exponent - 9)
    off = ((o - X).abs() - half).clamp(min=0).square().sum((1, 2)).sqrt()
    assert bool((off <= 2 * error).all()), (off / error).tolist()
    # and nowhere by more than 25 standard deviations of that
    assert float(((o - X).abs() - half).max()) <= 25 * float((2 * error).max()) / (r * c) ** 0.5
