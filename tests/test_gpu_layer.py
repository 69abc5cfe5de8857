"""The layer's operators on the GPU against their float64 definitions (layer_ref.py): every output
element within the bound derived there, at the sizes, masks and routings where they can go wrong,
and a whole layer forward and backward, eager and replayed from a captured graph."""

import gc

import numpy as np
import pytest
import torch

import combine_shuffling_amd as cs
import layer_ref as ref
import oracle
from combine_shuffling_amd import _abi

from gpu_util import say

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture
def big_tensors():
    """Gives the memory of a test of large tensors back, for the tests that follow."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def bf16(a, dev=None):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t if dev is None else t.to(dev)


def rounded(a):
    """float64 values of a rounded to bf16."""
    return bf16(a).double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    err = np.abs(got - want)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} elements outside; at {i}: "
                             f"{got[i]!r}, want {want[i]!r} +- {np.broadcast_to(bound, err.shape)[i]!r}")


def random_routing(rng, T, E, k, kind="uniform"):
    score = rng.random((T, E))
    if kind == "skewed":
        score += 2.0 * (np.arange(E) < max(1, E // 8)) + (np.arange(E) == 0)
    elif kind == "few":      # only the last k experts are used
        score += 9.0 * (np.arange(E) >= E - k)
    idx = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    if kind == "bad" and T > 0:
        for t in range(0, T, 3):
            idx[t, rng.integers(k)] = rng.choice([-1, E, 2 ** 30, -2 ** 31])
        for t in range(1, T, 4):
            idx[t, k - 1] = idx[t, 0]
    return idx


def routed(idx, E, R, H, dev, **kw):
    plan = cs.Plan(idx.shape[0], H, E, idx.shape[1], R, **kw)
    return plan.route(torch.from_numpy(idx).to(dev))


# ---- gradients of the shuffle

SHUFFLE = [
    # T, H, E, k, R, routing, plan
    (1, 8, 1, 1, 1, "uniform", {}),
    (3, 24, 4, 2, 2, "uniform", {}),
    (130, 520, 8, 2, 2, "bad", {}),
    (257, 512, 30, 8, 7, "uniform", {}),
    (61, 1032, 20, 5, 4, "skewed", {}),
    (40, 4104, 64, 16, 4, "uniform", {}),
    (33, 264, 1024, 11, 8, "bad", {}),
    (300, 64, 16, 4, 8, "uniform", dict(ranks_per_node=2, node_dedup=True)),
    (300, 64, 16, 4, 8, "bad", dict(ranks_per_node=2, node_dedup=True, load_aware_forwarders=True)),
    (1000, 64, 16, 4, 8, "uniform", dict(band_tokens=256)),
    (5000, 7168, 32, 8, 8, "uniform", {}),
]


def slots(plan, T, k):
    return plan.read("slot_of").reshape(T, k).astype(np.int64)


@pytest.mark.parametrize("T,H,E,k,R,kind,kw", SHUFFLE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_dispatch_backward(T, H, E, k, R, kind, kw, dtype, dev):
    say(f"[layer] dispatch backward T={T} H={H} E={E} k={k} {kind} {kw} {dtype}")
    rng = np.random.default_rng(T + H)
    plan = routed(random_routing(rng, T, E, k, kind), E, R, H, dev, **kw)
    g = rounded(rng.normal(size=(T * k, H)))
    full = torch.full((T + 2, H), 7.0, dtype=dtype, device=dev)
    out = plan.dispatch_backward(bf16(g, dev), full[:T], out_dtype=dtype)   # before any dispatch
    assert out.data_ptr() == full.data_ptr()
    want, mag = ref.dispatch_backward(g, slots(plan, T, k))
    err = k * U * mag
    check(out, want, err if dtype == torch.float32 else err + ref.BF16_HALF * (np.abs(want) + err)
          + ref.TINY, "grad_x")
    assert (full[T:] == 7).all()


@pytest.mark.parametrize("T,H,E,k,R,kind,kw", SHUFFLE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_combine_backward(T, H, E, k, R, kind, kw, dtype, dev):
    say(f"[layer] combine backward T={T} H={H} E={E} k={k} {kind} {kw} {dtype}")
    rng = np.random.default_rng(2 * T + H)
    plan = routed(random_routing(rng, T, E, k, kind), E, R, H, dev, **kw)
    y = rounded(rng.normal(size=(T * k, H)))
    g = rng.normal(size=(T, H)).astype(np.float32).astype(np.float64)
    if dtype == torch.bfloat16:
        g = rounded(g)
    w = rng.normal(size=(T, k)).astype(np.float32)
    gy = torch.full((T * k + 1, H), 7.0, dtype=torch.bfloat16, device=dev)
    got_y, got_w = plan.combine_backward(torch.from_numpy(g).to(dtype).to(dev), bf16(y, dev),
                                         torch.from_numpy(w).to(dev), grad_y=gy[: T * k])
    want_y, rows, want_w, mag = ref.combine_backward(g, y, w.astype(np.float64), slots(plan, T, k))
    want_y[~rows] = 7.0      # rows that no slot owns are left as they were
    check(got_y, want_y, (ref.BF16_HALF + 2 * U) * np.abs(want_y) + ref.TINY, "grad_y")
    check(got_w, want_w, H * U * mag, "grad_w")
    assert (gy[T * k:] == 7).all()


@pytest.mark.parametrize("kw", [{}, dict(ranks_per_node=2, node_dedup=True)], ids=["single", "dedup"])
def test_shuffle_gradients_are_the_adjoints(kw, dev):
    # Small integers, so that every sum is exact: <dispatch(x), g> = <x, dispatch_backward(g)> and
    # <combine(y, w), g> = <y, grad_y> = <w, grad_w>, to the last bit.
    rng = np.random.default_rng(9)
    T, H, E, k, R = 200, 264, 12, 3, 4
    plan = routed(random_routing(rng, T, E, k), E, R, H, dev, **kw)
    small = lambda *s: rng.integers(-2, 3, size=s).astype(np.float64)  # noqa: E731
    x, g, y, go = small(T, H), small(T * k, H), small(T * k, H), small(T, H)
    w = small(T, k)
    recv, _ = plan.dispatch(bf16(x, dev))
    gx = plan.dispatch_backward(bf16(g, dev), out_dtype=torch.float32)
    assert (f64(recv) * g).sum() == (x * f64(gx)).sum()
    wt = torch.from_numpy(w.astype(np.float32)).to(dev)
    out = plan.combine(bf16(y, dev), wt, out_dtype=torch.float32)
    gy, gw = plan.combine_backward(bf16(go, dev), bf16(y, dev), wt)
    want = (f64(out) * go).sum()
    assert (f64(gy) * y).sum() == want and (f64(gw) * w).sum() == want


# ---- the experts' products

ACTS = ["none", "relu", "silu", "gelu", "swiglu", "geglu"]
EXPERTS = [
    # T, E, k, K, N, routing
    (1, 1, 1, 8, 8, "uniform"),
    (1, 8, 2, 64, 64, "uniform"),
    (2, 40, 8, 136, 72, "uniform"),
    (16, 16, 4, 512, 256, "uniform"),
    (16, 200, 3, 1000, 40, "uniform"),
    (13, 6, 2, 2056, 24, "few"),
    (100, 60, 4, 96, 88, "skewed"),
    (63, 4, 2, 72, 200, "bad"),
    (65, 100, 6, 1000, 328, "uniform"),
    (300, 7, 3, 264, 520, "uniform"),
    (513, 5, 2, 88, 1032, "skewed"),
    (700, 12, 2, 1032, 264, "few"),
    (1100, 3, 2, 320, 384, "bad"),
    (40, 1024, 16, 64, 64, "uniform"),
]


def expert_inputs(rng, T, E, k, K, N, kind, act, integers=False):
    idx = random_routing(rng, T, E, k, kind)
    _, off = ref.layout(idx, E)
    Z = 2 * N if act in ref.KIND else N
    if integers:
        draw = lambda *s: rng.integers(-2, 3, size=s).astype(np.float64)  # noqa: E731
        return idx, off, draw(T * k, K), draw(E, Z, K), draw(E, Z), draw(T * k, N)
    x = rounded(rng.normal(size=(T * k, K)))
    w = rounded(rng.normal(size=(E, Z, K)) / np.sqrt(K))
    b = rng.normal(size=(E, Z)).astype(np.float32).astype(np.float64)
    return idx, off, x, w, b, rounded(rng.normal(size=(T * k, N)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,K,N,kind", EXPERTS)
def test_expert_linear(T, E, k, K, N, kind, act, dev):
    say(f"[layer] expert_linear T={T} E={E} k={k} K={K} N={N} {kind} {act}")
    rng = np.random.default_rng(T + K + N)
    idx, off, x, w, b, res = expert_inputs(rng, T, E, k, K, N, kind, act)
    plan = routed(idx, E, 1, 8, dev)
    rows, used = T * k, off[-1]
    xd, wd, rd = bf16(x, dev), bf16(w, dev), bf16(res, dev)
    bd = torch.from_numpy(b.astype(np.float32)).to(dev)
    for bias, residual, save in ((None, None, False), (bd, None, True), (bd, rd, True),
                                 (None, rd, False)):
        full = torch.full((rows + 1, N), 7.0, dtype=torch.bfloat16, device=dev)
        y, pre = plan.expert_linear(xd, wd, bias, residual, act, save, y=full[:rows])
        want, ey, z, ez = ref.expert_linear(x, w, None if bias is None else b,
                                            None if residual is None else res, act, off)
        check(y[:used], want[:used], ey[:used], f"y (bias {bias is not None}, residual "
              f"{residual is not None})")
        assert (full[used:] == 7).all(), "rows that no slot owns were written"
        assert (pre is not None) == save
        if save:
            check(pre[:used], z[:used], ez[:used], "pre")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,K,N,kind", EXPERTS)
def test_expert_linear_backward(T, E, k, K, N, kind, act, dev):
    say(f"[layer] expert_linear_backward T={T} E={E} k={k} K={K} N={N} {kind} {act}")
    rng = np.random.default_rng(T + 2 * K + N)
    idx, off, x, w, _, gy = expert_inputs(rng, T, E, k, K, N, kind, act)
    plan = routed(idx, E, 1, 8, dev)
    Z = w.shape[1]
    pre = rounded(rng.normal(size=(T * k, Z))) if act != "none" else None
    args = (bf16(gy, dev), bf16(x, dev), bf16(w, dev), None if pre is None else bf16(pre, dev), act)
    used = off[-1]
    want = ref.expert_linear_backward(gy[:used], x[:used], w, None if pre is None else pre[:used],
                                      act, off)
    for dtype in (torch.float32, torch.bfloat16):
        gx, gw, gb = plan.expert_linear_backward(*args, bias_grad=True, grad_w_dtype=dtype)
        check(gx[:used], *want["grad_x"], "grad_x")
        value, bound = want["grad_w"]
        if dtype == torch.bfloat16:
            bound = bound + ref.BF16_HALF * (np.abs(value) + bound) + ref.TINY
        check(gw, value, bound, f"grad_w {dtype}")
        check(gb, *want["grad_bias"], "grad_bias")
    # one at a time, the same bits
    for which in range(3):
        one = plan.expert_linear_backward(*args, x_grad=which == 0, w_grad=which == 1,
                                          bias_grad=which == 2)
        assert [t is not None for t in one] == [i == which for i in range(3)]
        want_t = (gx, gw, gb)[which]
        n = used if which == 0 else want_t.shape[0]
        assert torch.equal(one[which][:n], want_t[:n])


@pytest.mark.parametrize("T,E,k,K,N,kind", [(65, 9, 2, 136, 72, "uniform"),
                                            (600, 3, 2, 264, 520, "skewed"),
                                            (9, 20, 4, 1000, 128, "uniform")])
def test_expert_products_of_integers_are_exact(T, E, k, K, N, kind, dev):
    # Products and sums of small integers are exact in float32, whatever the order.
    rng = np.random.default_rng(K)
    idx, off, x, w, b, gy = expert_inputs(rng, T, E, k, K, N, kind, "none", integers=True)
    plan = routed(idx, E, 1, 8, dev)
    xd, wd, gd = bf16(x, dev), bf16(w, dev), bf16(gy, dev)
    y, _ = plan.expert_linear(xd, wd, torch.from_numpy(b.astype(np.float32)).to(dev))
    assert np.array_equal(f64(y), rounded(ref.product(x, w, b, off)[0]))
    gx, gw, gb = plan.expert_linear_backward(gd, xd, wd, bias_grad=True, grad_w_dtype=torch.float32)
    want = ref.expert_linear_backward(gy, x, w, None, "none", off)
    assert np.array_equal(f64(gx), rounded(want["grad_x"][0]))
    assert np.array_equal(f64(gw), want["grad_w"][0])
    assert np.array_equal(f64(gb), want["grad_bias"][0])


@pytest.mark.parametrize("T", [4, 37, 300])
def test_values_that_are_not_finite_stay_in_their_rows(T, dev):
    # One row of expert 1 is NaN and one of expert 2 infinite: other rows, and other experts'
    # weight gradients, are what they are without them.  Widths end inside a step.
    rng = np.random.default_rng(T)
    E, k, K, N = 4, 2, 72, 136
    idx, off, x, w, _, gy = expert_inputs(rng, T, E, k, K, N, "uniform", "none")
    plan = routed(idx, E, 1, 8, dev)
    wd = bf16(w, dev)
    clean = plan.expert_linear(bf16(x, dev), wd)[0], *plan.expert_linear_backward(
        bf16(gy, dev), bf16(x, dev), wd, bias_grad=True)
    hit = [off[1], off[2] + (off[3] - off[2]) // 2]
    assert off[1] < off[2] < off[3]
    x[hit[0]], gy[hit[0]] = np.nan, np.nan
    x[hit[1]], gy[hit[1]] = np.inf, -np.inf
    got = plan.expert_linear(bf16(x, dev), wd)[0], *plan.expert_linear_backward(
        bf16(gy, dev), bf16(x, dev), wd, bias_grad=True)
    rows = np.setdiff1d(np.arange(off[-1]), hit)
    for i in (0, 1):
        assert torch.equal(got[i][rows], clean[i][rows])
        assert not torch.isfinite(got[i][hit].float()).any()
    for i in (2, 3):
        for e in (0, 3):
            assert torch.equal(got[i][e], clean[i][e])
        assert torch.isnan(got[i][1].float()).all()


def test_empty_batch(dev):
    E, K, N = 5, 64, 40
    plan = cs.Plan(0, 64, E, 2, 1).route(torch.empty(0, 2, dtype=torch.int32, device=dev))
    none = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device=dev)  # noqa: E731
    w = torch.ones(E, N, K, dtype=torch.bfloat16, device=dev)
    assert plan.expert_linear(none(K), w)[0].shape == (0, N)
    gx, gw, gb = plan.expert_linear_backward(none(N), none(K), w, bias_grad=True)
    assert gx.shape == (0, K) and not gw.any() and not gb.any()
    assert plan.dispatch_backward(none(64)).shape == (0, 64)
    gy, gw = plan.combine_backward(none(64), none(64), torch.empty(0, 2, device=dev))
    assert gy.shape == (0, 64) and gw.shape == (0, 2)
    idx, wt = plan.router(torch.empty(0, E, device=dev))
    assert idx.shape == wt.shape == (0, 2)


@pytest.mark.parametrize("T,band,E,k,K,N,act", [
    (1000, 256, 6, 2, 136, 72, "swiglu"),     # bands that end inside the slots of bias sums
    (700, 256, 60, 3, 72, 264, "gelu"),
    (1300, 512, 3, 2, 264, 520, "none"),
    (260, 256, 40, 1, 64, 64, "silu"),        # a last band of fewer rows than experts
])
def test_expert_products_on_banded_plans(T, band, E, k, K, N, act, dev):
    say(f"[layer] banded experts T={T} band={band} E={E} k={k} K={K} N={N} {act}")
    rng = np.random.default_rng(T + N)
    idx, _, x, w, b, gy = expert_inputs(rng, T, E, k, K, N, "uniform", act)
    idx[5, 0] = -1          # a dropped slot: the band's last row stays as it is
    plan = routed(idx, E, 1, 64, dev, band_tokens=band)
    Z = w.shape[1]
    pre = rounded(rng.normal(size=(T * k, Z))) if act != "none" else None
    xd, wd, gd = bf16(x, dev), bf16(w, dev), bf16(gy, dev)
    full = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=dev)
    y, _ = plan.expert_linear(xd, wd, torch.from_numpy(b.astype(np.float32)).to(dev), None, act, y=full)
    gx, gw, gb = plan.expert_linear_backward(gd, xd, wd, None if pre is None else bf16(pre, dev), act,
                                             bias_grad=True, grad_w_dtype=torch.float32)
    offs = plan.read("expert_offsets").reshape(-1, E + 1)
    assert np.array_equal(offs[:, 0], np.arange(len(offs)) * band * k)
    total = {n: [0.0, 0.0] for n in ("grad_w", "grad_bias")}
    for o in offs:
        s = slice(o[0], o[-1])
        local = o - o[0]
        want, ey, _, _ = ref.expert_linear(x[s], w, b, None, act, local)
        check(y[s], want, ey, "y")
        r = ref.expert_linear_backward(gy[s], x[s], w, None if pre is None else pre[s], act, local)
        check(gx[s], *r["grad_x"], "grad_x")
        for n, t in total.items():
            t[0], t[1] = t[0] + r[n][0], t[1] + r[n][1]
    # the bands' sums are added up in float32: their number more roundings of the magnitudes
    for n, got in (("grad_w", gw), ("grad_bias", gb)):
        check(got, total[n][0], total[n][1] * (1 + len(offs)), n)
    hole = offs[0][-1]
    assert hole == band * k - 1 and (y[hole] == 7).all()


# ---- the router

ROUTER = [
    # T, E, k, R, G, nodes
    (1, 1, 1, 1, 1, 0),
    (5, 8, 2, 2, 2, 0),
    (129, 64, 8, 4, 4, 0),
    (70, 65, 6, 7, 7, 0),
    (100, 256, 8, 64, 8, 4),
    (33, 100, 6, 10, 2, 3),      # five nodes of 20
    (50, 30, 4, 8, 2, 2),        # nodes of 8, 8, 7, 7
    (20, 64, 1, 64, 1, 1),       # 64 nodes of one expert
    (9, 1024, 16, 4, 4, 0),
    (40, 300, 16, 3, 3, 0),
    (300, 16, 16, 1, 1, 0),      # every expert
    # tokens that share a wave
    (4099, 64, 8, 8, 8, 0),
    (4097, 100, 6, 10, 2, 3),
    (5003, 30, 16, 30, 2, 8),    # 15 nodes of 2
    (4101, 256, 8, 64, 8, 4),
    (4100, 130, 5, 18, 3, 2),    # nodes of 24, 22, 21, 21, 21 and 21
    (4098, 200, 4, 20, 1, 2),    # more nodes than lanes: a wave each
]


def nodes_of_experts(E, R, G):
    lo = oracle.expert_partition(E, R)
    return [next(r for r in range(R) if lo[r] <= e < lo[r + 1]) // G for e in range(E)]


@pytest.mark.parametrize("T,E,k,R,G,nodes", ROUTER)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("how", ["plain", "bias", "masked", "huge"])
def test_router(T, E, k, R, G, nodes, dtype, how, dev):
    say(f"[layer] router T={T} E={E} k={k} nodes={nodes} {dtype} {how}")
    rng = np.random.default_rng(T + E)
    rows = np.arange(T) % 301   # large batches repeat rows, so that the definition has few to do
    x = torch.from_numpy(rng.normal(size=(min(T, 301), E)).astype(np.float32) * 2)
    if how == "masked":       # rows that a mask leaves nothing of, or less than k; NaN; infinity
        x[rng.random(x.shape) < 0.6] = -np.inf
        x[0] = -np.inf
        if T > 4:
            x[1], x[2, E // 2], x[3, ::2], x[4, E - 1] = float("nan"), float("nan"), np.inf, np.inf
            x[2, E // 3] = torch.finfo(torch.bfloat16).min
    if how == "huge":         # far from 0, where exp over- and underflows
        x = x * 40 - 60
    few = x.to(dtype)
    x = few[rows]
    bias = rng.normal(size=E).astype(np.float32) if how == "bias" else None
    plan = cs.Plan(T, 8, E, k, R, G)
    xd = x.to(dev)
    values = x.double().numpy()
    node_of = nodes_of_experts(E, R, G)
    want = ref.router_choice(few.float().numpy(), bias, k, node_of, nodes)[rows]
    gw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            bd = None if bias is None else torch.from_numpy(bias).to(dev)
            idx, w = plan.router(xd, bd, score, renorm, 2.5, nodes)
            assert np.array_equal(idx.cpu().numpy(), want), (score, renorm)
            ww = ref.router_weights(values, want, score, renorm, 2.5)
            # exp of x - max: its argument rounds once (|x - max| u in the result), exp and the
            # sums of up to E terms a few u; subnormal results flush by at most 2^-126
            with np.errstate(invalid="ignore"):
                spread = np.abs(values - values.max(1, keepdims=True))
            spread = np.minimum(np.nan_to_num(spread, nan=0.0, posinf=0.0, neginf=0.0), 100).max()
            rel = (16 + E + 4 * spread) * U
            check(w, ww, rel * ww + 2.5 * 2.0 ** -120, f"w {score} {renorm}")
            gl = plan.router_backward(xd, idx, gw.to(dev), score, renorm, 2.5)
            g = gw.double().numpy()
            wl = ref.router_backward(values, want, g, score, renorm, 2.5)
            size = 2.5 * (np.abs(g).max(1, keepdims=True) + np.abs(g).sum(1, keepdims=True))
            bound = 4 * rel * size + 2.0 ** -120
            if dtype == torch.bfloat16:
                bound = bound + ref.BF16_HALF * (np.abs(wl) + bound)
            check(gl, wl, np.broadcast_to(bound, wl.shape), f"grad {score} {renorm}")


def test_router_ties_go_to_the_lowest_id(dev):
    for E, k in ((8, 3), (256, 8), (1000, 16)):
        plan = cs.Plan(4, 8, E, k, 1)
        x = torch.zeros(4, E, device=dev)
        x[1] = -0.0
        x[2, ::2] = -0.0
        x[3] = float("-inf")
        idx, w = plan.router(x)
        assert (idx == torch.arange(k, device=dev)).all()
        assert (w[:3] == 1 / k).all() and (w[3] == 0).all()


def test_router_backward_takes_foreign_ids(dev):
    # an id out of range adds nothing, one that is there twice adds both
    plan = cs.Plan(2, 8, 6, 3, 1)
    x = torch.randn(2, 6, device=dev)
    idx = torch.tensor([[1, 1, 4], [-1, 7, 2]], dtype=torch.int32, device=dev)
    gw = torch.tensor([[1.0, 2.0, 4.0], [8.0, 16.0, 32.0]], device=dev)
    got = plan.router_backward(x, idx, gw, "sigmoid", False, 1.0).cpu()
    s = torch.sigmoid(x.cpu().double())
    want = torch.zeros(2, 6, dtype=torch.float64)
    want[0, 1], want[0, 4], want[1, 2] = 3.0, 4.0, 32.0
    assert ((got - want * s * (1 - s)).abs() <= 64 * U * want).all()


# ---- together

class Layer:
    """One Mixture-of-Experts layer with a gated first product: forward, then every gradient."""

    def __init__(self, T, H, I, E, k, R, dev, seed, **kw):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rand = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=dev) * scale  # noqa: E731
        self.plan = cs.Plan(T, H, E, k, R, **kw)
        self.logits = rand(T, E)
        self.bias = rand(E, scale=0.2)
        self.x = rand(T, H).bfloat16()
        self.w1 = rand(E, 2 * I, H, scale=H ** -0.5).bfloat16()
        self.b1 = rand(E, 2 * I)
        self.w2 = rand(E, H, I, scale=I ** -0.5).bfloat16()
        self.grad_out = rand(T, H).bfloat16()

    def step(self):
        p = self.plan
        idx, w = cs.router(p, self.logits, self.bias, scale=1.5)
        p.route(idx)
        recv, _ = cs.dispatch(p, self.x)
        h, pre = cs.expert_linear(p, recv, self.w1, self.b1, activation="swiglu", save_pre=True)
        y, _ = cs.expert_linear(p, h, self.w2)
        out = cs.combine(p, y, w)
        grad_y, grad_w = cs.combine_backward(p, self.grad_out, y, w)
        grad_h, grad_w2, _ = cs.expert_linear_backward(p, grad_y, h, self.w2)
        grad_recv, grad_w1, grad_b1 = cs.expert_linear_backward(p, grad_h, recv, self.w1, pre,
                                                                "swiglu", bias_grad=True)
        grad_x = cs.dispatch_backward(p, grad_recv)
        grad_logits = cs.router_backward(p, self.logits, idx, grad_w, scale=1.5)
        return dict(idx=idx, w=w, recv=recv, h=h, pre=pre, y=y, out=out, grad_y=grad_y, grad_w=grad_w,
                    grad_h=grad_h, grad_w2=grad_w2, grad_recv=grad_recv, grad_w1=grad_w1,
                    grad_b1=grad_b1, grad_x=grad_x, grad_logits=grad_logits)


@pytest.mark.parametrize("T,kw", [(1, {}), (77, {}), (500, dict(ranks_per_node=1, node_dedup=True))])
def test_layer_step_by_step(T, kw, dev):
    # Every operator's output against its definition on the GPU's own inputs to it.
    H, I, E, k, R = 136, 72, 10, 3, 5
    m = Layer(T, H, I, E, k, R, dev, seed=T, **kw)
    s = m.step()
    v = {n: f64(t) for n, t in s.items()}
    idx = s["idx"].cpu().numpy()
    assert np.array_equal(idx, ref.router_choice(m.logits.cpu().numpy(), m.bias.cpu().numpy(), k,
                                                 [0] * E, 0))
    slot, off = ref.layout(idx, E)
    assert np.array_equal(v["recv"][slot], np.repeat(f64(m.x)[:, None], k, 1))
    w1, w2, b1 = f64(m.w1), f64(m.w2), f64(m.b1)
    want, ey, z, ez = ref.expert_linear(v["recv"], w1, b1, None, "swiglu", off)
    check(s["h"], want, ey, "h")
    check(s["pre"], z, ez, "pre")
    want, ey, _, _ = ref.expert_linear(v["h"], w2, None, None, "none", off)
    check(s["y"], want, ey, "y")
    gy, _, gw, mag = ref.combine_backward(f64(m.grad_out), v["y"], v["w"], slot)
    check(s["grad_y"], gy, (ref.BF16_HALF + 2 * U) * np.abs(gy) + ref.TINY, "grad_y")
    check(s["grad_w"], gw, H * U * mag, "grad_w")
    half = lambda x, b: b + ref.BF16_HALF * (np.abs(x) + b) + ref.TINY  # noqa: E731
    r = ref.expert_linear_backward(v["grad_y"], v["h"], w2, None, "none", off)
    check(s["grad_h"], *r["grad_x"], "grad_h")
    check(s["grad_w2"], r["grad_w"][0], half(*r["grad_w"]), "grad_w2")
    r = ref.expert_linear_backward(v["grad_h"], v["recv"], w1, v["pre"], "swiglu", off)
    check(s["grad_recv"], *r["grad_x"], "grad_recv")
    check(s["grad_w1"], r["grad_w"][0], half(*r["grad_w"]), "grad_w1")
    check(s["grad_b1"], *r["grad_bias"], "grad_b1")
    gx, mag = ref.dispatch_backward(v["grad_recv"], slot)
    check(s["grad_x"], gx, half(gx, k * U * mag), "grad_x")


def same(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])]


def test_layer_in_a_graph_and_on_another_stream(dev):
    # Two layers captured into two graphs, replayed in turn between eager steps of both.
    layers = [Layer(300, 264, 136, 12, 4, 3, dev, seed=i) for i in range(2)]
    eager = [m.step() for m in layers]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layers[0].step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert same(eager[0], other) == []
    graphs, outs = [], []
    for m in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step())
        graphs.append(g)
    for i in range(4):
        for j in (0, 1):
            for t in outs[j].values():
                t.zero_()
            graphs[j].replay()
            if i % 2:
                torch.cuda.synchronize()
            again = layers[1 - j].step()
            assert same(eager[1 - j], again) == []
            torch.cuda.synchronize()
            assert same(eager[j], outs[j]) == [], (i, j)


def test_products_captured_on_their_own(dev):
    # Small plans leave the offsets' scan to the first call that needs them.  One that is only
    # recorded into a graph does not count for eager calls, and a graph replayed after another
    # route of the plan uses that route.
    rng = np.random.default_rng(2)
    T, E, k, K, N = 90, 7, 2, 72, 136
    idx, _, x, w, _, _ = expert_inputs(rng, T, E, k, K, N, "uniform", "none")
    other = random_routing(rng, T, E, k, "skewed")
    xd, wd = bf16(x, dev), bf16(w, dev)
    routes = [torch.from_numpy(i).to(dev) for i in (idx, other)]
    want = [cs.Plan(T, 8, E, k, 1).route(i).expert_linear(xd, wd)[0] for i in routes]
    assert not torch.equal(*want)
    plan = cs.Plan(T, 8, E, k, 1).route(routes[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = plan.expert_linear(xd, wd)
        again, _ = plan.expert_linear(xd, wd)
    assert torch.equal(plan.expert_linear(xd, wd)[0], want[0])
    for i in (0, 1, 0, 1):
        plan.route(routes[i])
        y.zero_()
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(again, want[i])
        assert torch.equal(plan.expert_linear(xd, wd)[0], want[i])


def test_outputs_and_workspace_given(dev):
    m = Layer(40, 72, 64, 6, 2, 1, dev, seed=4)
    s = m.step()
    p = m.plan
    args = (s["grad_h"], s["recv"], m.w1, s["pre"], "swiglu")
    outs = [torch.empty_like(s[n]) for n in ("grad_recv", "grad_w1", "grad_b1")]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    got = cs.expert_linear_backward(p, *args, bias_grad=True, grad_x=outs[0], grad_w=outs[1],
                                    grad_bias=outs[2], workspace=ws)
    for o, g, n in zip(outs, got, ("grad_recv", "grad_w1", "grad_b1")):
        assert o.data_ptr() == g.data_ptr() and torch.equal(o, s[n])
    with pytest.raises(ValueError, match="grad_w"):
        cs.expert_linear_backward(p, *args, grad_w=outs[1].float())
    with pytest.raises(cs.MoeError):      # a workspace that is not 256-byte aligned
        cs.expert_linear_backward(p, *args, workspace=ws[16:])


def test_given_stream_is_used(dev):
    # The calls run on the stream they are given, after what is queued there.
    m = Layer(64, 64, 64, 8, 2, 1, dev, seed=1)
    want = m.step()
    side = torch.cuda.Stream()
    x = torch.zeros_like(m.x)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(50):
            x.add_(1)
        x.copy_(want["recv"][:64])
        recv = torch.cat([x, want["recv"][64:]])
    h, _ = m.plan.expert_linear(recv, m.w1, m.b1, activation="swiglu", stream=side)
    gx = m.plan.dispatch_backward(want["grad_recv"], stream=side)
    idx, w = m.plan.router(m.logits, m.bias, scale=1.5, stream=side)
    side.synchronize()
    assert torch.equal(h, want["h"]) and torch.equal(gx, want["grad_x"])
    assert torch.equal(idx, want["idx"]) and torch.equal(w, want["w"])


def test_timing_names_every_launch(dev):
    names = set()
    for T in (4, 300):   # few rows an expert, and many
        m = Layer(T, 264, 136, 12, 4, 3, dev, seed=5)
        m.plan.timing(64)
        s = m.step()
        for which in (dict(x_grad=False, bias_grad=True), dict(w_grad=False)):
            m.plan.expert_linear_backward(s["grad_y"], s["h"], m.w2, **which)
        names |= {n for n, _, ms in m.plan.timing_read() if ms > 0}
        m.plan.timing(0)
    assert {_abi.kernel_name(i) for i in range(22, _abi.KERNEL_COUNT)} <= names


@pytest.mark.slow
def test_offsets_past_32_bits(dev, big_tensors):
    # Rows whose elements pass 2^31 (and byte offsets 2^32): the last rows against their values.
    T, k, E, H, N = 70000, 8, 16, 4096, 8
    rng = np.random.default_rng(0)
    idx = random_routing(rng, T, E, k)
    plan = routed(idx, E, 1, H, dev)
    slot = slots(plan, T, k)
    assert T * k * H > 2 ** 31
    x = torch.randint(-2, 3, (T, H), device=dev, generator=None).bfloat16()
    recv, _ = plan.dispatch(x)
    w = torch.randint(-1, 2, (E, N, H), device=dev).bfloat16()
    y, _ = plan.expert_linear(recv, w)
    off = plan.read("expert_offsets")
    tail = slice(T * k - 500, T * k)
    want = recv[tail].float() @ w[E - 1].float().t()
    assert off[E - 1] < T * k - 500 and torch.equal(y[tail], want.bfloat16())
    gy = torch.randint(-1, 2, (T * k, N), device=dev).bfloat16()
    gx, gw, _ = plan.expert_linear_backward(gy, recv, w, grad_w_dtype=torch.float32)
    assert torch.equal(gx[tail], (gy[tail].float() @ w[E - 1].float()).bfloat16())
    last = slice(int(off[E - 1]), T * k)
    assert torch.equal(gw[E - 1], (gy[last].double().t() @ recv[last].double()).float())
    gt = plan.dispatch_backward(recv, out_dtype=torch.float32)
    assert torch.equal(gt, x.float() * k)
    grad_y, gwt = plan.combine_backward(x, recv, torch.ones(T, k, device=dev))
    assert torch.equal(grad_y, recv)
    assert torch.equal(gwt, (x.float() ** 2).sum(1, keepdim=True).expand(T, k))
    assert slot.max() == T * k - 1


@pytest.mark.slow
def test_most_rows(dev, big_tensors):
    # The most tokens that the 32-bit row indices allow, one expert and rows of 16 bytes: token t's
    # row is row t.
    T = 2 ** 31 - 4098
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 * (1 << 30):
        pytest.skip("needs about 180 GiB of free device memory")
    plan = cs.Plan(T, 8, 1, 1, 1)
    plan.route(torch.zeros(T, 1, dtype=torch.int32, device=dev))
    y = torch.empty(T, 8, dtype=torch.bfloat16, device=dev)
    part = 1 << 26
    for a in range(0, T, part):
        b = min(T, a + part)
        y[a:b] = ((torch.arange(a, b, device=dev)[:, None] * 8 + torch.arange(8, device=dev)) % 7 - 3)
    g = torch.full((T, 8), 2.0, dtype=torch.bfloat16, device=dev)
    g[T - 5:] = 1.0
    w = torch.full((T, 1), 0.5, device=dev)
    gx = plan.dispatch_backward(y)
    for a in range(0, T, part):
        assert torch.equal(gx[a: a + part], y[a: a + part]), a
    gy, gw = plan.combine_backward(g, y, w, grad_y=gx)
    for a in range(0, T, part):
        s = slice(a, a + part)
        assert torch.equal(gy[s], 0.5 * g[s]), a
        assert torch.equal(gw[s], (g[s].float() * y[s].float()).sum(1, keepdim=True)), a
