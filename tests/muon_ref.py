"""The matrix step in 64 bits, and a model of the orthogonalisation's roundings. Nothing here
comes from the library: numpy only, written from the formulas.
"""
from __future__ import annotations

import numpy as np

COEF = (3.4445, -4.7750, 2.0315)


def triples(coefficients, steps):
    c = COEF if coefficients is None else coefficients
    return [tuple(c)] * steps if np.ndim(c) == 1 else [tuple(t) for t in c]


def orthogonalize(x, *, steps=5, coefficients=None, eps=1e-7, scale=1.0):
    """[R, C] in 64 bits."""
    X = np.asarray(x, np.float64)
    X = X / (np.sqrt((X * X).sum()) + eps)
    for a, b, c in triples(coefficients, steps):
        if X.shape[0] > X.shape[1]:
            A = X.T @ X
            X = a * X + X @ (b * A + c * A @ A)
        else:
            A = X @ X.T
            X = a * X + (b * A + c * A @ A) @ X
    return scale * X


def _half(v):
    """fp16 of 1024 v, as the value that it stands for."""
    return (v * np.float32(1024)).astype(np.float16).astype(np.float32) / np.float32(1024)


def _split(X):
    """X as hi, fp16 of 4096 X with ties away from zero, and X again with 8 more bits."""
    v = X * np.float32(4096)
    v = np.where(np.abs(v) < 2.0 ** -14, np.float32(0), v)
    t = v.view(np.uint32) + np.uint32(1 << 12)
    hi = (t & np.uint32(0xFFFFE000)).view(np.float32)
    x = ((t & np.uint32(0xFFFFFFE0)) - np.uint32(1 << 12)).view(np.float32)
    zero = v == 0
    return [np.where(zero, np.float32(0), w) / np.float32(4096) for w in (hi, x)]


def model(x, *, steps=5, coefficients=None, eps=1e-7, scale=1.0):
    """The same with the roundings that the kernels make before o's own: fp16 operands, fp32
    sums and diagonals, X with 18 bits. In fp32; its sums are in another order."""
    X = np.asarray(x, np.float64)
    tall = X.shape[0] > X.shape[1]
    X = (X / (np.sqrt((X * X).sum()) + eps)).astype(np.float32)
    if tall:
        X = np.ascontiguousarray(X.T)
    for k, (a, b, c) in enumerate(triples(coefficients, steps)):
        a, b, c = np.float32(a), np.float32(b), np.float32(c)
        hi, X = _split(X)
        A = hi @ hi.T
        d = np.diagonal(A).copy()
        np.fill_diagonal(A, 0)
        F = _half(A)
        FF = F @ F
        e = b * d + c * (d * d + np.diagonal(FF))
        G = b * F + c * (FF + (d[:, None] + d[None, :]) * F)
        np.fill_diagonal(G, 0)
        X = a * X + e[:, None] * (X if steps - 1 - k <= 2 else hi) + _half(G) @ hi
    X = np.float32(scale) * X
    return X.T if tall else X


# What the kernels may differ from the formula by. They make the model's roundings, each to
# the other side now and then as their sums run in another order, so their errors are of the
# model's size; four times its largest error is allowed at every element, and twice its
# norm over all, beside o's own rounding (2^-8 of the value at most).
def bounds(x, **kw):
    want = orthogonalize(x, **kw)
    off = model(x, **kw) - want
    return want, 2.0 ** -8 * np.abs(want) + 4 * np.abs(off).max() + 2.0 ** -133, \
        2.0 ** -8 * np.linalg.norm(want) + 2 * np.linalg.norm(off)


def momentum(g, m, mu, nesterov):
    """(m', u) in fp32, one operation at a time."""
    mu = np.float32(mu)
    m2 = mu * m + g
    return m2, g + mu * m2 if nesterov else m2


def update(p, o, lr, weight_decay):
    return p * np.float32(1.0 - lr * weight_decay) - np.float32(lr) * o
