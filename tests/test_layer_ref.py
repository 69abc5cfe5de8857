"""The layer's float64 reference (CPU): its gradients against central differences of its forward
functions, and its layout against the oracle's route plan."""

import numpy as np
import pytest

import layer_ref as ref
import oracle

H = 1e-5      # central differences: error about H^2 (third derivatives of order 1) + 1e-16 / H
TOL = 1e-8


def differences(f, x):
    out = np.zeros_like(x)
    flat, g = x.reshape(-1), out.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + H
        a = f()
        flat[i] = keep - H
        b = f()
        flat[i] = keep
        g[i] = (a - b) / (2 * H)
    return out


def routing(T, E, k, seed):
    rng = np.random.default_rng(seed)
    return np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)


@pytest.mark.parametrize("T,E,k,R", [(1, 1, 1, 1), (37, 8, 3, 3), (64, 30, 4, 8)])
def test_layout_is_the_oracles(T, E, k, R):
    idx = routing(T, E, k, T)
    p = oracle.route_plan(idx, E, R, R)
    slot, off = ref.layout(idx, E)
    assert np.array_equal(slot, p["slot_of"])
    assert np.array_equal(off, p["expert_offsets"])


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "swiglu", "geglu"])
def test_expert_gradient_against_differences(kind):
    rng = np.random.default_rng(3)
    T, E, k, K, N = 5, 3, 2, 4, 3
    _, off = ref.layout(routing(T, E, k, 1), E)
    Z = 2 * N if kind in ref.KIND else N
    x, w, b = rng.normal(size=(T * k, K)), rng.normal(size=(E, Z, K)), rng.normal(size=(E, Z))
    gy = rng.normal(size=(T * k, N))

    def loss():
        return float((ref.expert_linear(x, w, b, None, kind, off)[0] * gy).sum())

    pre, _ = ref.product(x, w, b, off)
    got = ref.expert_linear_backward(gy, x, w, pre, kind, off)
    for name, v in (("grad_x", x), ("grad_w", w), ("grad_bias", b)):
        assert np.abs(got[name][0] - differences(loss, v)).max() < TOL, name


def test_shuffle_gradients_against_differences():
    rng = np.random.default_rng(4)
    T, E, k, D = 6, 5, 2, 3
    idx = routing(T, E, k, 2)
    idx[3, 1] = idx[3, 0]      # a dropped slot
    slot, _ = ref.layout(idx, E)
    y, w = rng.normal(size=(T * k, D)), rng.normal(size=(T, k))
    x, g = rng.normal(size=(T, D)), rng.normal(size=(T, D))
    valid = (slot >= 0)[:, :, None]

    def combine():
        return float((np.where(valid, w[:, :, None] * y[np.maximum(slot, 0)], 0).sum(1) * g).sum())

    gy, rows, gw, _ = ref.combine_backward(g, y, w, slot)
    assert np.abs(gy - differences(combine, y)).max() < TOL
    assert np.abs(gw - differences(combine, w)).max() < TOL
    assert rows.sum() == T * k - 1
    gr = rng.normal(size=(T * k, D))

    def dispatch():
        return float(sum((x[t] * gr[s]).sum() for t in range(T) for s in slot[t] if s >= 0))

    assert np.abs(ref.dispatch_backward(gr, slot)[0] - differences(dispatch, x)).max() < TOL


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_router_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 7))
    idx = ref.router_choice(x.astype(np.float32), None, 3, [0] * 7, 0)
    gw = rng.normal(size=(4, 3))

    def loss():
        return float((ref.router_weights(x, idx, score, renormalise, 1.7) * gw).sum())

    got = ref.router_backward(x, idx, gw, score, renormalise, 1.7)
    assert np.abs(got - differences(loss, x)).max() < TOL


def test_router_choice_ties_masks_and_nodes():
    nan, inf = float("nan"), float("inf")
    x = np.array([[1, 1, 1, 1], [nan, -inf, nan, -inf], [inf, 0, inf, 1], [-0.0, 0.0, -1, -2]],
                 dtype=np.float32)
    got = ref.router_choice(x, None, 3, [0] * 4, 0)
    assert got.tolist() == [[0, 1, 2], [1, 3, 0], [0, 2, 3], [0, 1, 2]]
    # two nodes of two: node 0 is worth 1 + 1, node 1 2 + (-3)
    y = np.array([[1, 1, 2, -3]], dtype=np.float32)
    assert ref.router_choice(y, None, 2, [0, 0, 1, 1], 1).tolist() == [[0, 1]]
    assert ref.router_weights(np.full((1, 4), -inf), np.array([[0, 1]]), "softmax", True, 1).tolist() \
        == [[0.0, 0.0]]
