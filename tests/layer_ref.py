"""The layer operators in 64 bits, with a bound on what fp32 sums and one rounding
may differ by. Nothing here comes from the library: numpy only, written from the
formulas; the generator is Philox4x32-10 as published.
"""
from __future__ import annotations

import numpy as np

ACTS = ("none", "relu", "gelu", "silu")
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}      # half a step, relative to the value
TINY = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149}


def philox(counter, key, rounds=10):
    """Philox4x32: counter is four uint64 arrays of 32-bit words, key two ints."""
    u = np.uint64
    low = u(0xFFFFFFFF)
    c = [np.asarray(x, dtype=u) for x in counter]
    k0, k1 = key
    for _ in range(rounds):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & low, (a >> u(32)) ^ c[3] ^ u(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def drop_factor(rows, cols, p, seed, offset):
    """[rows, cols] factors: 0 where dropped, 65536 / (65536 - thr) elsewhere."""
    return _factors(np.arange(rows, dtype=np.uint64), cols, p, seed, offset)


def drop_row(row, cols, p, seed, offset):
    """The factors of one row."""
    return _factors(np.array([row], dtype=np.uint64), cols, p, seed, offset)[0]


def _factors(rows, cols, p, seed, offset):
    thr = int(np.rint(p * 65536))
    if thr == 0:
        return np.ones((len(rows), cols))
    g = (cols + 7) // 8
    i, j = np.meshgrid(rows, np.arange(g, dtype=np.uint64), indexing="ij")
    offset &= (1 << 64) - 1
    full = np.ones_like(i)
    w = philox((j, i, full * np.uint64(offset & 0xFFFFFFFF), full * np.uint64(offset >> 32)),
               (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    draws = np.empty((len(rows), g, 8), dtype=np.uint64)
    for k in range(8):
        draws[:, :, k] = (w[k // 2] >> np.uint64(16 * (k % 2))) & np.uint64(0xFFFF)
    keep = draws.reshape(len(rows), 8 * g)[:, :cols] >= thr
    return keep * (65536.0 / (65536.0 - thr))


def act(name, z):
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "gelu":
            return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1 + np.exp(-z))
    return z


def slope(name, z):
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "relu":
            return np.where(z > 0, 1.0, 0.0)
        if name == "gelu":
            c = np.sqrt(2 / np.pi)
            h = np.clip(z, -1e3, 1e3)
            t = np.tanh(c * (h + 0.044715 * h ** 3))
            return 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * c * (1 + 3 * 0.044715 * h * h)
        if name == "silu":
            h = np.clip(z, -700, 700)
            g = 1 / (1 + np.exp(-h))
            return g * (1 + h * (1 - g))
    return np.ones_like(z)


# A sum of n products, in any order and with any grouping in fp32, is off by at most
# n * 2^-23 of the sum of their magnitudes (each of n - 1 additions rounds a partial
# sum that is at most that sum, by 2^-24 of it; the matrix instruction may truncate
# where it adds, which is twice that; bf16 products are exact in fp32).
def sum_err(n, mags):
    return (n + 4) * 2.0 ** -23 * mags


# The activations are z * logistic(a(z)): the hardware's exp2 and reciprocal and the
# argument's rounding are off by at most 2^-24 * (2 |argument| + 8) relative, where
# the logistic is not yet 0; arguments beyond 90 give 0 or 1 to fp32. 200 * 2^-24 < 2^-16
# bounds the relative error, and where the argument is large the value is below
# e^-|argument|, so that the absolute error stays below 2^-20 * max(1, |z|).
def act_err(z):
    return 2.0 ** -20 * np.maximum(1.0, np.abs(z))


# d act / dz is at most 1.13 (GELU) and 1.10 (SiLU); a slope is off by 2^-18 at most
# (the logistic's relative error times the polynomial in front of it, |h| * 2c *
# (1 + 3 a h^2) * s (1 - s) <= 1.2 and its terms below 4).
LIPSCHITZ = 1.13
SLOPE_ERR = 2.0 ** -18


def rounded(y, out):
    return U[out] * np.abs(y) + TINY[out]


def linear_forward(x, w, bias=None, *, act_name="none", p=0.0, seed=0, offset=0, residual=None, out="bf16"):
    """x [M, K], w [N, K] (float64). Returns (y, bound on y, z, bound on z)."""
    M, K = x.shape
    z = x @ w.T
    mags = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + bias
        mags = mags + np.abs(bias)
    ez = sum_err(K + 1, mags)
    f = drop_factor(M, w.shape[0], p, seed, offset)
    h = act(act_name, z)
    eh = ez * (LIPSCHITZ if act_name != "none" else 1.0) + (act_err(z) if act_name in ("gelu", "silu") else 0.0)
    y = np.where(f == 0, 0.0, h * f)
    ey = np.where(f == 0, 0.0, eh * f + 2.0 ** -23 * np.abs(y))
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -24 * (np.abs(y) + ey)
    ey = ey * (1 + U[out]) + rounded(y, out)
    return y, ey, z, ez * (1 + U["bf16"]) + rounded(z, "bf16")


def linear_grad_input(dz, w, *, act_name="none", z=None, p=0.0, seed=0, offset=0, out="bf16"):
    M, N = dz.shape
    d = dz @ w
    e = sum_err(N, np.abs(dz) @ np.abs(w))
    f = drop_factor(M, w.shape[1], p, seed, offset)
    s = slope(act_name, z) if act_name != "none" else np.ones_like(d)
    y = np.where(f == 0, 0.0, d * f * s)
    e = e * f * np.abs(s) + np.abs(d) * f * (SLOPE_ERR if act_name in ("gelu", "silu") else 0.0)
    e = np.where(f == 0, 0.0, e + 2.0 ** -22 * np.abs(y))
    return y, e * (1 + U[out]) + rounded(y, out)


def linear_grad_weight(dz, x, *, old=None, out="bf16"):
    """[N, K] gradient; old [N, K]."""
    M = dz.shape[0]
    g = dz.T @ x
    e = sum_err(M, np.abs(dz).T @ np.abs(x))
    if old is not None:
        g = g + old
        e = e + 2.0 ** -24 * (np.abs(g) + e)
    return g, e * (1 + U[out]) + rounded(g, out)


def column_sums(dz, *, old=None, out="bf16"):
    g = dz.sum(0)
    e = sum_err(dz.shape[0], np.abs(dz).sum(0))
    if old is not None:
        g = g + old
        e = e + 2.0 ** -24 * (np.abs(g) + e)
    return g, e * (1 + U[out]) + rounded(g, out)


def dropout_add(x, *, p, seed, offset, residual=None, out="bf16"):
    f = drop_factor(x.shape[0], x.shape[1], p, seed, offset)
    y = np.where(f == 0, 0.0, x * f)
    e = 2.0 ** -23 * np.abs(y)
    if residual is not None:
        y = y + residual
        e = e + 2.0 ** -24 * (np.abs(y) + e)
    return y, e * (1 + U[out]) + rounded(y, out)


def dropout_grad(dy, *, p, seed, offset, act_name="none", z=None, out="bf16"):
    f = drop_factor(dy.shape[0], dy.shape[1], p, seed, offset)
    s = slope(act_name, z) if act_name != "none" else np.ones_like(dy)
    y = np.where(f == 0, 0.0, dy * f * s)
    e = np.abs(dy) * f * (SLOPE_ERR if act_name in ("gelu", "silu") else 0.0) + 2.0 ** -22 * np.abs(y)
    return y, e * (1 + U[out]) + rounded(y, out)
