"""Plain float64 definitions of the layer's operators (numpy, no code of the library), and the
error bounds the GPU results are held to.

Bounds.  u = 2^-24.  A float32 sum of n products of bf16 values differs from the exact one by at
most n * 2u * S, S the sum of the magnitudes (each addition rounds once, by at most half a step
under round-to-nearest and one step if the matrix cores truncate).  Rounding a value v to bf16
moves it by at most 2^-8 |v| (half a step), or half the smallest subnormal.
"""

from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8
TINY = 2.0 ** -133   # the smallest bf16 subnormal
KIND = {"swiglu": "silu", "geglu": "gelu"}
# Largest slopes of the activations, and of their derivatives (|gelu''| <= 0.80, |silu''| <= 0.5).
SLOPE = 1.13
CURVE = 0.80

_erf = np.vectorize(math.erf)


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def phi(z):
    return 0.5 * (1 + _erf(z / math.sqrt(2.0))) if np.size(z) else z


def act(kind, z):
    kind = KIND.get(kind, kind)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z * sigmoid(z)
    if kind == "gelu":
        return z * phi(z)
    return z


def slope(kind, z):
    kind = KIND.get(kind, kind)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = sigmoid(z)
        return s + z * s * (1 - s)
    if kind == "gelu":
        return phi(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


def layout(idx, E):
    """(slot_of [T, k], expert offsets [E + 1]) of the receive layout; -1 where the id is out of
    range or repeated."""
    T, k = idx.shape
    ok = np.zeros((T, k), dtype=bool)
    for t in range(T):
        seen = set()
        for j in range(k):
            e = int(idx[t, j])
            ok[t, j] = 0 <= e < E and e not in seen
            seen.add(e)
    slot = np.full((T, k), -1, dtype=np.int64)
    off = [0]
    for e in range(E):
        at = np.argwhere(ok & (idx == e))   # tokens ascending
        for i, (t, j) in enumerate(at):
            slot[t, j] = off[-1] + i
        off.append(off[-1] + len(at))
    return slot, np.array(off)


# ---- the shuffle's gradients

def dispatch_backward(grad_recv, slot):
    """(grad_x, sum of magnitudes)"""
    g = np.where((slot >= 0)[:, :, None], grad_recv[np.maximum(slot, 0)], 0.0)
    return g.sum(1), np.abs(g).sum(1)


def combine_backward(grad_out, y, w, slot):
    """(grad_y, rows written, grad_w, sum of magnitudes of grad_w)"""
    rows = np.zeros(y.shape[0], dtype=bool)
    grad_y = np.zeros_like(y)
    grad_w = np.zeros(w.shape)
    mag = np.zeros(w.shape)
    for j in range(w.shape[1]):
        at = np.nonzero(slot[:, j] >= 0)[0]
        s = slot[at, j]
        rows[s] = True
        grad_y[s] = w[at, j: j + 1] * grad_out[at]
        p = grad_out[at] * y[s]
        grad_w[at, j] = p.sum(1)
        mag[at, j] = np.abs(p).sum(1)
    return grad_y, rows, grad_w, mag


# ---- the experts' products

def product(x, w, bias, off):
    """(z, error bound of its float32 value)"""
    rows, K = x.shape
    z = np.zeros((rows, w.shape[1]))
    mag = np.zeros_like(z)
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        z[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
        if bias is not None:
            z[a:b] += bias[e]
            mag[a:b] += np.abs(bias[e])
    return z, (K + 2) * 2 * U * mag


def expert_linear(x, w, bias, residual, kind, off):
    """(y, bound of y, z, bound of pre)"""
    z, ez = product(x, w, bias, off)
    n = z.shape[1]
    if kind in KIND:
        n //= 2
        g, up = z[:, :n], z[:, n:]
        a = act(kind, g)
        y = a * up
        ey = SLOPE * ez[:, :n] * (np.abs(up) + ez[:, n:]) + np.abs(a) * ez[:, n:]
    else:
        y = act(kind, z)
        ey = SLOPE * ez
    ey = ey + 16 * U * np.abs(y)           # evaluating the activation: a few float32 roundings
    if kind in ("silu", "gelu", "swiglu", "geglu"):
        ey = ey + 256 * U * np.abs(y)      # exp and erfc: relative error of the hardware's exp2
    if residual is not None:
        y = y + residual
        ey = ey + 2 * U * np.abs(y)
    return y, ey + BF16_HALF * (np.abs(y) + ey) + TINY, z, ez + BF16_HALF * (np.abs(z) + ez) + TINY


def expert_grad_z(gy, pre, kind):
    """(grad_z, error bound of its float32 value)"""
    if kind == "none":
        return gy, np.zeros_like(gy)
    n = gy.shape[1]
    if kind in KIND:
        g, up = pre[:, :n], pre[:, n:]
        gz = np.concatenate([gy * up * slope(kind, g), gy * act(kind, g)], 1)
        size = np.concatenate([np.abs(gy * up) * (1 + np.abs(g)), np.abs(gy * g)], 1)
    else:
        gz = gy * slope(kind, pre)
        size = np.abs(gy) * (1 + np.abs(pre))
    return gz, 64 * U * size


def expert_linear_backward(gy, x, w, pre, kind, off):
    """Dict of (value, bound) for grad_x, grad_w (float32) and grad_bias."""
    gz, ez = expert_grad_z(gy, pre, kind)
    eb = ez if kind == "none" else ez + BF16_HALF * (np.abs(gz) + ez) + TINY  # as bf16 operand
    gx, gw = np.zeros((x.shape[0], w.shape[2])), np.zeros(w.shape)
    gb = np.zeros(w.shape[:2])
    ex, ew, ebias = np.zeros_like(gx), np.zeros_like(gw), np.zeros_like(gb)
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        gx[s] = gz[s] @ w[e]
        ex[s] = eb[s] @ np.abs(w[e]) + (w.shape[1] + 1) * 2 * U * ((np.abs(gz[s]) + eb[s]) @ np.abs(w[e]))
        gw[e] = gz[s].T @ x[s]
        ew[e] = eb[s].T @ np.abs(x[s]) + (n + 1) * 2 * U * ((np.abs(gz[s]) + eb[s]).T @ np.abs(x[s]))
        gb[e] = gz[s].sum(0)
        ebias[e] = ez[s].sum(0) + (n + 1) * U * (np.abs(gz[s]) + ez[s]).sum(0)
    ex = ex + BF16_HALF * (np.abs(gx) + ex) + TINY
    return {"grad_x": (gx, ex), "grad_w": (gw, ew), "grad_bias": (gb, ebias)}


# ---- the router

def router_choice(logits, bias, k, node_of, nodes_per_token):
    """ids [T, k].  logits: float32 [T, E]; the keys are float32 sums by definition; a NaN key
    ranks below -infinity."""
    T, E = logits.shape
    key = logits.astype(np.float32) + (bias if bias is not None else np.float32(0))
    out = np.zeros((T, k), dtype=np.int32)
    for t in range(T):
        def rank(v):
            return (1, 0.0) if math.isnan(v) else (0, -float(v))
        allowed = list(range(E))
        if nodes_per_token:
            worth = []
            for n in range(max(node_of) + 1):
                v = sorted((key[t, e] for e in range(E) if node_of[e] == n),
                           key=lambda q: rank(q))[:2]
                v = [np.float32(-np.inf) if math.isnan(q) else q for q in v]
                worth.append(v[0] if len(v) == 1 or v[0] == np.inf else np.float32(v[0] + v[1]))
            kept = sorted(range(len(worth)), key=lambda n: (rank(worth[n]), n))[:nodes_per_token]
            allowed = [e for e in allowed if node_of[e] in kept]
        out[t] = sorted(allowed, key=lambda e: (rank(key[t, e]), e))[:k]
    return out


def _shares(v):
    """exp(v - max) / sum over the last axis: infinities share, all -infinity gives 0."""
    m = v.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(v == -np.inf, 0.0, np.where(v == m, 1.0, np.exp(v - m)))
    s = e.sum(-1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def _log_score(x, score):
    return x if score == "softmax" else np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))


def router_weights(logits, idx, score, renormalise, scale):
    x = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    if renormalise:
        return scale * _shares(_log_score(np.take_along_axis(x, idx, 1), score))
    p = _shares(x) if score == "softmax" else sigmoid(x)
    return scale * np.take_along_axis(p, idx, 1)


def router_backward(logits, idx, grad_w, score, renormalise, scale):
    x = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    T, k = idx.shape
    out = np.zeros_like(x)
    g = scale * grad_w
    xs = np.take_along_axis(x, idx, 1)
    if renormalise:
        p = _shares(_log_score(xs, score))
        d = p * (g - (p * g).sum(1, keepdims=True))
        if score == "sigmoid":
            d = d * sigmoid(-xs)
    elif score == "softmax":
        full = _shares(x)
        p = np.take_along_axis(full, idx, 1)
        out -= full * (p * g).sum(1, keepdims=True)
        d = p * g
    else:
        d = g * sigmoid(xs) * sigmoid(-xs)
    for t in range(T):
        for j in range(k):
            out[t, idx[t, j]] += d[t, j]
    return out
