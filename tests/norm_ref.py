"""A norm's rows and their gradient in 64 bits, with bounds on what fp32 arithmetic and one
rounding may differ by. Nothing here comes from the library: numpy only, written from the
formulas.

u = 2^-24 bounds the relative error of one fp32 operation. A lane adds at most ceil(N / 512)
chunks of eight columns one after another (fewer where more waves share a row), then 6
steps join a wave and at most 8 more its row: a sum over a row has at most
DEPTH(N) = 8 ceil(N / 512) + 14 additions in a chain, and is off by at most that times u times
the sum of magnitudes (Higham, Accuracy and Stability, 4.2), to first order; the factor
1.01 covers the higher ones.
"""
from __future__ import annotations

import numpy as np

from layer_ref import U, rounded

u = 2.0 ** -24


def depth(N):
    return 8 * -(-N // 512) + 14


def row_sum(v, err):
    """Mean over each row of what is off by err, in fp32: (mean, bound)."""
    N = v.shape[1]
    m = v.sum(1, keepdims=True) / N
    mag = (np.abs(v) + err).sum(1, keepdims=True) / N
    return m, 1.01 * (err.sum(1, keepdims=True) / N + (depth(N) + 2) * u * mag)


def forward(s, w, b, *, rms, eps, out):
    """s [M, N] as stored. Returns (y, bound, stats [M, 2], bound)."""
    M, N = s.shape
    zero = np.zeros_like(s)
    mean, em = (np.zeros((M, 1)), np.zeros((M, 1))) if rms else row_sum(s, zero)
    d = s - mean
    ed = em + u * (np.abs(d) + em)
    var, ev = row_sum(d * d, 2 * np.abs(d) * ed + ed * ed)
    eps32 = float(np.float32(eps))
    ev = ev + u * (var + ev + eps32) + abs(eps32 - eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = (var + eps) ** -0.5
        # the square root and the quotient round once each
        er = np.maximum((np.maximum(var - ev, 0) + eps) ** -0.5 - r, r - (var + ev + eps) ** -0.5) * (1 + 3 * u) + 3 * u * r
        t = d * r
        et = ed * r + np.abs(d) * er + ed * er + u * np.abs(t)
        y = t * w + b
        ey = np.abs(w) * et * (1 + u) + u * np.abs(t * w) + u * (np.abs(y) + np.abs(w) * et)
    ey = 1.01 * ey
    return y, ey * (1 + U[out]) + rounded(y, out), np.hstack((mean, r)), 1.01 * np.hstack((em, er))


def grad(dy, x, w, stats, *, rms, res=None, out="bf16", old_w=None, old_b=None, grad_out="f32"):
    """Returns ((dx, bound), (dw, bound), (db, bound)) for the stats that the call is given."""
    M, N = dy.shape
    mean, r = stats[:, :1], stats[:, 1:]
    h = (x - mean) * r
    eh = 2.01 * u * np.abs(h)
    g = dy * w
    eg = u * np.abs(g)
    mg, emg = (np.zeros((M, 1)), np.zeros((M, 1))) if rms else row_sum(g, eg)
    mgh, emgh = row_sum(g * h, np.abs(g) * eh + eg * np.abs(h) + u * np.abs(g * h))
    inner = g - mg - h * mgh
    ei = eg + emg + np.abs(h) * emgh + eh * (np.abs(mgh) + emgh) + 2 * u * (np.abs(g) + np.abs(mg) + np.abs(h * mgh))
    dx = r * inner
    ex = np.abs(r) * ei
    if res is not None:
        dx = dx + res
    ex = 1.01 * (ex + u * np.abs(dx))
    got = [(dx, ex * (1 + U[out]) + rounded(dx, out))]
    for v, e, old in ((dy * h, np.abs(dy) * eh, old_w), (dy, np.zeros_like(dy), old_b)):
        s = v.sum(0)
        es = e.sum(0) + 1.01 * (M + 8) * u * (np.abs(v) + e).sum(0)
        if old is not None:
            s = s + old
            es = es + u * (np.abs(s) + es)
        got.append((s, es * (1 + U[grad_out]) + rounded(s, grad_out)))
    return got
