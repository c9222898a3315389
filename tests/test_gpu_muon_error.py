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
