"""Plain float64 definitions of the operators of moe_block.h (numpy, no code of the library), and
the error bounds the GPU results are held to.  u = 2^-24, half a step of float32 relative to the
value; sums of float32 values in a tree of depth d are off by at most d u S, S the sum of the
magnitudes.
"""

from __future__ import annotations

import numpy as np

import layer_ref as ref
from layer_ref import BF16_HALF, TINY, U

# A row's sum: at most 16 values a lane in order, 6 folds over the lanes, 16 waves, and a factor 1 / H
# that is rounded itself and in the product.
DEPTH = 16 + 6 + 16 + 2


def stored(value, bound, dtype):
    """Bound of a value after rounding to "bf16" or "f32"."""
    half, tiny = (BF16_HALF, TINY) if dtype == "bf16" else (U, 2.0 ** -149)
    return bound + half * (np.abs(value) + bound) + tiny


def norm(x, gamma, beta, rms, eps):
    """Dict of (value, bound) for y (before rounding), mean and rstd ([T])."""
    n = x.shape[1]
    if rms:
        mean, em = np.zeros(len(x)), np.zeros(len(x))
    else:
        mean = x.mean(1)
        em = DEPTH * U * np.abs(x).sum(1) / n
    d = x - mean[:, None]
    ed = em[:, None] + U * (np.abs(d) + em[:, None])
    var = (d * d).mean(1)
    ev = (2 * np.abs(d) * ed + ed * ed).mean(1)
    ev = ev + DEPTH * U * (var + ev) + U * (var + eps)
    v = var + eps
    with np.errstate(divide="ignore"):
        rstd = 1 / np.sqrt(v)
        er = np.maximum(1 / np.sqrt(np.maximum(v - ev, eps)) - rstd, rstd - 1 / np.sqrt(v + ev))
    er = er + 3 * U * (rstd + er)
    a, r, e = np.abs(d), rstd[:, None], er[:, None]
    h = d * r
    eh = ed * (r + e) + a * e
    eh = eh + U * (np.abs(h) + eh)
    y = h * gamma + beta
    ey = eh * np.abs(gamma)
    ey = ey + 2 * U * (np.abs(h * gamma) + np.abs(beta) + ey)
    return {"y": (y, ey), "mean": (mean, em + 2.0 ** -149), "rstd": (rstd, er)}


def norm_backward(gy, x, stats, gamma, gtotal, rms):
    """Dict of (value, bound) for grad_x (before rounding), grad_gamma and grad_beta; stats: the
    float32 values that the kernel reads."""
    n, T = x.shape[1], x.shape[0]
    mean, rstd = stats[:, :1], stats[:, 1:]
    h = (x - mean) * rstd
    eh = 3 * U * np.abs(h)
    g = gy * gamma
    along = (g * h).mean(1, keepdims=True)
    ea = (DEPTH + 6) * U * np.abs(g * h).mean(1, keepdims=True)
    s = np.zeros_like(along) if rms else g.mean(1, keepdims=True)
    es = np.zeros_like(along) if rms else (DEPTH + 2) * U * np.abs(g).mean(1, keepdims=True)
    inner = g - s - h * along
    size = np.abs(g) + np.abs(s) + np.abs(h * along)
    e = es + np.abs(h) * ea + eh * (np.abs(along) + ea) + 4 * U * size
    gx = rstd * inner
    eg = np.abs(rstd) * e + 2 * U * np.abs(gx)
    if gtotal is not None:
        gx = gx + gtotal
        eg = eg + U * (np.abs(gx) + eg)
    return {"grad_x": (gx, eg),
            "grad_gamma": ((gy * h).sum(0), (T + 5) * U * np.abs(gy * h).sum(0)),
            "grad_beta": (gy.sum(0), T * U * np.abs(gy).sum(0))}
