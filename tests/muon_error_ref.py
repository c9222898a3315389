"""How far an orthogonalisation in 32 bits may be from the formula, by arithmetic, and a model
of pairs of fp16 numbers. Nothing here comes from the library: numpy only.

An iterate is kept, and an operand read, to 2^-23 of its value (a pair of fp16 numbers: 11 bits
of hi, 11 of lo and lo's sign; fp32 is 2^-24); a product leaves out lo lo, 2^-22 of each of its terms
at most, and its sums are fp32. The roundings of different elements are independent, so that
together they are to a matrix's norm what each is to its element: a step
X' = a X + b A X + c A A X of norm-wise roundings of 2^-23 in each of its terms leaves at most
    fresh = 2^-23 (|a| + |b| s^2 + |c| s^4) |X|,   s the largest singular value of X,
and the first X one of 2^-23 |X|. What an earlier step has left is multiplied by the derivative of
the step, whose norm is at most g, the largest |p'| between 0 and s of p(s) = a s + b s^3 + c s^5:
that is a where X holds nothing. To first order, then,
    error <= sum over steps of fresh times the g of those behind it,
and twice that is allowed. (The model of muon_ref.py, with fp16 operands and 18 bits of X, has fewer
bits than the kernels, and its bounds are wide.)
"""
from __future__ import annotations

import numpy as np

import muon_ref as R


def growth(x, *, steps=5, coefficients=None, eps=1e-7, scale=1.0):
    """(the formula's result in 64 bits, the norm of what may be added to it before it is rounded)."""
    X = np.asarray(x, np.float64)
    X = X / (np.sqrt((X * X).sum()) + eps)
    X = X.T if X.shape[0] > X.shape[1] else X
    error = 2.0 ** -23 * np.linalg.norm(X)
    for a, b, c in R.triples(coefficients, steps):
        A = X @ X.T
        s = np.sqrt(max(np.linalg.eigvalsh(A)[-1], 0.0))
        at = np.linspace(0, s, 200)
        error = error * np.abs(a + 3 * b * at ** 2 + 5 * c * at ** 4).max()
        error += 2.0 ** -23 * (abs(a) + abs(b) * s ** 2 + abs(c) * s ** 4) * np.linalg.norm(X)
        X = a * X + (b * A + c * A @ A) @ X
    want = scale * X
    return want.T if np.shape(x)[0] > np.shape(x)[1] else want, 2 * abs(scale) * error


def beyond_rounding(o, want):
    """The norm of what o, in bf16, is off by beyond half a step of its own: at most that of what
    was off before the rounding."""
    most = np.maximum(np.abs(o), np.abs(want))
    half = np.exp2(np.floor(np.log2(np.maximum(most, 2.0 ** -126))) - 8)
    return float(np.linalg.norm(np.maximum(np.abs(o - want) - half, 0.0)))


def check(o, x, name=None, **kw):
    """o [B, R, C] against the formula for x (numpy, 64 bits)."""
    for k in range(o.shape[0]):
        want, allowed = growth(x[k], **kw)
        off = beyond_rounding(o[k], want)
        assert off <= allowed, (name, k, off / np.linalg.norm(want), allowed / np.linalg.norm(want))


def _pair(v, by):
    t = (v * np.float32(by)).astype(np.float32)
    hi = t.astype(np.float16).astype(np.float32)
    lo = (t - hi).astype(np.float16).astype(np.float32)
    return hi / np.float32(by), lo / np.float32(by)


def _product(a, b):
    """a b^T of two pairs, without lo lo."""
    return np.concatenate([a[0], a[0], a[1]], 1) @ np.concatenate([b[0], b[1], b[0]], 1).T


def model(x, *, steps=5, coefficients=None, eps=1e-7, scale=1.0):
    """The iteration with X, A and b A + c A A in pairs of fp16 numbers of 4096 and 1024 times their
    values, and diagonals and sums in fp32."""
    f = np.float32
    X = np.asarray(x, np.float64)
    tall = X.shape[0] > X.shape[1]
    X = (X / (np.sqrt((X * X).sum()) + eps)).astype(f)
    X = np.ascontiguousarray(X.T) if tall else X
    for a, b, c in R.triples(coefficients, steps):
        a, b, c = f(a), f(b), f(c)
        px = _pair(X, 4096)
        A = _product(px, px)
        d = np.diagonal(A).copy()
        np.fill_diagonal(A, 0)
        pa = _pair(A, 1024)
        A = pa[0] + pa[1]
        FF = _product(pa, pa)
        e = b * d + c * (d * d + np.diagonal(FF))
        G = b * A + c * (FF + (d[:, None] + d[None, :]) * A)
        np.fill_diagonal(G, 0)
        X = (a + e[:, None]) * (px[0] + px[1]) + _product(_pair(G, 1024), tuple(np.ascontiguousarray(v.T) for v in px))
    X = f(scale) * X
    return X.T if tall else X


def matrix(kind, rows, cols, rng):
    """equalK: K equal singular values; rankK: of K normal directions; fall: from 1 to 1e-5."""
    def directions(k):
        return [np.linalg.qr(rng.standard_normal((n, k)))[0] for n in (rows, cols)]
    if kind.startswith("equal"):
        q = directions(int(kind[5:]))
        return q[0] @ q[1].T
    if kind.startswith("rank"):
        k = int(kind[4:])
        return rng.standard_normal((rows, k)) @ rng.standard_normal((k, cols))
    if kind == "fall":
        q = directions(min(rows, cols))
        return (q[0] * np.logspace(0, -5, min(rows, cols))) @ q[1].T
    return rng.standard_normal((rows, cols))


# kinds of spectrum at sizes and step counts; the a's of the default coefficients multiply to 485
# in five steps, 1,670 in six and 5,752 in seven
CASES = [("equal64", 128, 512, 5), ("equal64", 512, 128, 5), ("equal66", 128, 256, 5), ("rank32", 64, 197, 5),
         ("rank32", 197, 64, 5), ("rank1", 128, 128, 5), ("rank1", 768, 768, 5), ("rank1", 8, 8, 5), ("rank6", 200, 200, 5),
         ("normal", 512, 512, 5), ("normal", 300, 130, 5), ("normal", 8, 8, 5), ("fall", 150, 150, 5),
         ("equal64", 128, 512, 6), ("rank1", 128, 128, 6), ("rank1", 128, 700, 7), ("rank1", 768, 128, 7),
         ("rank6", 200, 200, 7), ("equal64", 128, 512, 7), ("fall", 150, 150, 7), ("normal", 140, 140, 3)]
# a published table that starts with larger gains
TABLE = [(8.28721201814563, -23.595886519098837, 17.300387312530933),
         (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
         (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
         (3.3184196573706015, -2.488488024314874, 0.51004894012372),
         (2.300652019954817, -1.6689039845747493, 0.4188073119525673)]

# (batch, rows, columns) whose products are cut in every way there is: tests/c/orth_plans.cpp
# prints how, tests/test_muon_plan.py holds that none is missing
PLAN_SIZES = [(1, 65, 70), (1, 67, 64), (1, 70, 12552), (1, 1835, 9244), (1, 2924, 2844), (1, 12659, 65), (2, 8470, 969),
              (3, 67, 8558), (3, 8840, 64), (6, 2449, 2309), (8, 1961, 2224), (8, 2008, 1956), (12, 513, 580),
              (12, 558, 521), (12, 774, 883), (12, 786, 785), (12, 1029, 1277), (12, 1047, 1041), (12, 1614, 2193),
              (1, 11008, 4096), (1, 4096, 11008)]
