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


# ---- 4-bit weights

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
INT4 = np.arange(16) - 8.0


def bytes_of(codes):
    """codes [E, Z, K] (0..15) as a checkpoint holds them: two a byte, the lower nibble first."""
    return (codes[:, :, 0::2] | codes[:, :, 1::2] << 4).astype(np.uint8)


def values4(codes, scales, fmt, group):
    """(weights, scale of each weight) [E, Z, K] in float64.  scales: float64 values (int4) or E8M0
    bytes (e2m1)."""
    s = scales if fmt == "int4" else np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    s = np.repeat(s, group, axis=2)[:, :, : codes.shape[2]]
    return (INT4 if fmt == "int4" else E2M1)[codes] * s, s


def quantize4(w, fmt, group):
    """(codes, scales) of bf16 values w [E, Z, K] (finite), by exact comparisons."""
    E, Z, K = w.shape
    n = -(-K // group)
    full = np.zeros((E, Z, n * group))
    full[:, :, :K] = w
    full = full.reshape(E, Z, n, group)
    amax = np.abs(full).max(3)
    if fmt == "int4":
        a = (amax.astype(np.float32) / np.float32(7)).astype(np.float32)
        bits = a.view(np.uint32).astype(np.uint64)
        bits = (bits + 0x7fff + ((bits >> 16) & 1)) >> 16 << 16      # to bf16, nearest even
        s = bits.astype(np.uint32).view(np.float32).astype(np.float64)
        with np.errstate(divide="ignore", invalid="ignore"):
            v = (full.astype(np.float32) / s[..., None].astype(np.float32)).astype(np.float64)
        v = np.where(s[..., None] > 0, np.clip(np.rint(v), -8, 7), 0)
        codes, scales = v.astype(int) + 8, s
    else:
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.ceil(np.log2(amax / 6)), 0).astype(int)
        # the smallest with amax <= 6 * 2^e, exactly
        e = np.where((amax > 0) & (amax <= 6 * np.ldexp(1.0, e - 1)), e - 1, e)
        e = np.where((amax > 0) & (amax > 6 * np.ldexp(1.0, e)), e + 1, e)
        e = np.where(amax > 0, np.clip(e, -127, 127), 0)
        v = full / np.ldexp(1.0, e)[..., None]
        m = np.abs(v)[..., None]
        d = np.abs(m - E2M1[:8])
        d = d + 1e-9 * (np.arange(8) % 2)                            # ties to the even code
        codes, scales = d.argmin(-1) + 8 * np.signbit(full), e + 127
    return codes.reshape(E, Z, -1)[:, :, :K], scales


def expert_linear4(x, codes, scales, fmt, group, bias, residual, kind, off):
    """(y, bound of y).  The products of INT4 codes are added up as products with 128 + c and
    with -136, so that their roundings are of sums of magnitude |x| (264 + c) times the scale."""
    w, s = values4(codes, scales, fmt, group)
    rows, K = x.shape
    z = np.zeros((rows, w.shape[1]))
    e = np.zeros_like(z)
    for i in range(len(off) - 1):
        a, b = off[i], off[i + 1]
        z[a:b] = x[a:b] @ w[i].T
        mag = np.abs(x[a:b]) @ np.abs(w[i]).T
        e[a:b] = (K + 8) * 2 * U * mag
        if fmt == "int4":
            e[a:b] += (2 * group + 2) * 2 * U * (np.abs(x[a:b]) @ (np.abs(s[i]) * (264 + codes[i])).T)
        if bias is not None:
            z[a:b] += bias[i]
            e[a:b] += 2 * U * (np.abs(z[a:b]) + np.abs(bias[i]))
    n = z.shape[1]
    if kind in ref.KIND:
        n //= 2
        g, up = z[:, :n], z[:, n:]
        y = ref.act(kind, g) * up
        ey = ref.SLOPE * e[:, :n] * (np.abs(up) + e[:, n:]) + np.abs(ref.act(kind, g)) * e[:, n:]
    else:
        y = ref.act(kind, z)
        ey = ref.SLOPE * e
    ey = ey + (16 if kind in ("none", "relu") else 272) * U * np.abs(y)   # as for bf16 weights
    if residual is not None:
        y = y + residual
        ey = ey + 2 * U * np.abs(y)
    return y, stored(y, ey, "bf16")
