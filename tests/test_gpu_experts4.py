"""The experts' products with 4-bit weights on the GPU against their float64 definitions
(block_ref.py): packing, quantizing, and every output element within the bound derived there."""

import numpy as np
import pytest
import torch

import block_ref
import combine_shuffling_amd as cs
import layer_ref as ref
from combine_shuffling_amd import _abi

from gpu_util import say
from test_gpu_layer import bf16, check, f64, random_routing, rounded, routed

pytestmark = pytest.mark.gpu

FORMATS = [("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32)]
IDS = [f"{f}-{g}" for f, g in FORMATS]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def draw(rng, E, Z, K, fmt, group, exact=False):
    """(codes, scales) as block_ref takes them; exact: scales are powers of two near 1."""
    codes = rng.integers(0, 16, size=(E, Z, K))
    shape = (E, Z, -(-K // group))
    if fmt == "e2m1":
        return codes, rng.integers(126, 129, size=shape)
    if exact:
        return codes, np.ldexp(1.0, rng.integers(-1, 2, size=shape))
    return codes, rounded(rng.normal(size=shape) / np.sqrt(K))     # of either sign


def packed(codes, scales, fmt, group, dev):
    s = bf16(scales, dev) if fmt == "int4" else torch.from_numpy(scales.astype(np.uint8)).to(dev)
    return cs.pack_experts4(torch.from_numpy(block_ref.bytes_of(codes)).to(dev), s, fmt, group)


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("E,Z,K", [(1, 8, 8), (3, 24, 40), (2, 40, 128), (5, 16, 136), (4, 264, 1000),
                                   (1, 8, 2056), (700, 8, 72)])
def test_packed_weights_are_the_values(E, Z, K, fmt, group, dev):
    say(f"[experts4] pack {E} x {Z} x {K} {fmt} {group}")
    rng = np.random.default_rng(Z + K)
    codes, scales = draw(rng, E, Z, K, fmt, group)
    if fmt == "e2m1":
        scales[rng.random(scales.shape) < 0.2] = 255       # NaN
        scales[rng.random(scales.shape) < 0.1] = 0         # the smallest, in whose place 2^-128 is subnormal
        scales[rng.random(scales.shape) < 0.1] = 252
    w4 = packed(codes, scales, fmt, group, dev)
    want, _ = block_ref.values4(codes, scales, fmt, group)
    got = f64(w4.values())
    assert np.array_equal(got, want.astype(np.float32), equal_nan=True)
    assert torch.equal(w4.values(torch.bfloat16).nan_to_num(), w4.values().bfloat16().nan_to_num())


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("E,Z,K", [(1, 8, 8), (3, 24, 40), (2, 40, 128), (4, 264, 1000)])
def test_quantizer(E, Z, K, fmt, group, dev):
    say(f"[experts4] quantize {E} x {Z} x {K} {fmt} {group}")
    rng = np.random.default_rng(Z + 2 * K)
    w = rng.normal(size=(E, Z, K)) * np.exp2(rng.integers(-20, 20, size=(E, Z, 1)))
    w[:, 1] = rng.integers(-12, 13, size=(E, K)) / 2       # ties
    w[:, 2] = 0
    w[:, 3, : K // 2] = 0
    w[:, 4] *= 2.0 ** -90
    w[:, 5] = rounded(w[:, 5] * 2.0 ** -110)
    w[:, 6] = np.sign(w[:, 6]) * 1e38
    w = rounded(w)
    codes, scales = block_ref.quantize4(w, fmt, group)
    want, _ = block_ref.values4(codes, scales, fmt, group)
    got = f64(cs.quantize_experts4(bf16(w, dev), fmt, group).values())
    assert np.array_equal(got, want.astype(np.float32))
    # a group with an infinity or a NaN is NaN, the others are what they were
    bad = w.copy()
    bad[0, 7, 0], bad[0, 0, K - 1] = np.inf, np.nan
    got = f64(cs.quantize_experts4(bf16(bad, dev), fmt, group).values())
    hit = np.zeros(w.shape, dtype=bool)
    hit[0, 7, : min(group, K)] = True
    hit[0, 0, (K - 1) // group * group:] = True
    assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], want[~hit].astype(np.float32))


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


def inputs(rng, T, E, k, K, N, kind, act, fmt, group, exact=False):
    idx = random_routing(rng, T, E, k, kind)
    _, off = ref.layout(idx, E)
    Z = 2 * N if act in ref.KIND else N
    codes, scales = draw(rng, E, Z, K, fmt, group, exact)
    if exact:
        ints = lambda *s: rng.integers(-2, 3, size=s).astype(np.float64)  # noqa: E731
        return idx, off, ints(T * k, K), codes, scales, ints(E, Z), ints(T * k, N)
    x = rounded(rng.normal(size=(T * k, K)))
    b = rng.normal(size=(E, Z)).astype(np.float32).astype(np.float64)
    return idx, off, x, codes, scales, b, rounded(rng.normal(size=(T * k, N)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("T,E,k,K,N,kind", EXPERTS)
def test_expert_linear4(T, E, k, K, N, kind, fmt, group, act, dev):
    say(f"[experts4] product T={T} E={E} k={k} K={K} N={N} {kind} {act} {fmt} {group}")
    rng = np.random.default_rng(T + K + N)
    idx, off, x, codes, scales, b, res = inputs(rng, T, E, k, K, N, kind, act, fmt, group)
    plan = routed(idx, E, 1, 8, dev)
    rows, used = T * k, off[-1]
    w4 = packed(codes, scales, fmt, group, dev)
    xd, rd, bd = bf16(x, dev), bf16(res, dev), torch.from_numpy(b.astype(np.float32)).to(dev)
    for bias, residual in ((None, None), (bd, rd)):
        full = torch.full((rows + 1, N), 7.0, dtype=torch.bfloat16, device=dev)
        y = plan.expert_linear4(xd, w4, bias, residual, act, y=full[:rows])
        want, ey = block_ref.expert_linear4(x, codes, scales, fmt, group, None if bias is None else b,
                                            None if residual is None else res, act, off)
        check(y[:used], want[:used], ey[:used], f"y (bias {bias is not None})")
        assert (full[used:] == 7).all(), "rows that no slot owns were written"


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("T,E,k,K,N,kind", [(1, 3, 1, 264, 40, "uniform"), (16, 16, 4, 1000, 72, "uniform"),
                                            (65, 9, 2, 136, 72, "uniform"),
                                            (600, 3, 2, 264, 520, "skewed"),
                                            (130, 20, 4, 1000, 128, "uniform"),
                                            (4000, 5, 2, 392, 776, "skewed")])
def test_products_of_integers_are_exact(T, E, k, K, N, kind, fmt, group, dev):
    # Products and sums of small integers and halves, under scales that are powers of two, are exact
    # in float32, whatever the order: every code, place and scale counts.
    say(f"[experts4] exact T={T} E={E} k={k} K={K} N={N} {kind} {fmt} {group}")
    rng = np.random.default_rng(K)
    idx, off, x, codes, scales, b, res = inputs(rng, T, E, k, K, N, kind, "none", fmt, group, True)
    plan = routed(idx, E, 1, 8, dev)
    y = plan.expert_linear4(bf16(x, dev), packed(codes, scales, fmt, group, dev),
                            torch.from_numpy(b.astype(np.float32)).to(dev), bf16(res, dev))
    w, _ = block_ref.values4(codes, scales, fmt, group)
    z = np.concatenate([x[off[e]: off[e + 1]] @ w[e].T + b[e] for e in range(E)])
    assert np.array_equal(f64(y), rounded(z + res[: off[-1]]))


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("T,E,k,K,N,kind", [
    (1, 6, 2, 7168, 40, "uniform"),      # few strips: eight waves share each
    (16, 16, 2, 7168, 72, "uniform"),    # x of 4 rows at a time in LDS
    (16, 2, 2, 7168, 24, "uniform"),     # of 16 rows, the contraction in phases
    (30, 4, 3, 3000, 136, "uniform"),    # of 16 rows, two phases of unequal length
    (3, 3, 1, 33000, 16, "uniform"),
    (40, 2, 2, 5000, 136, "uniform"),    # passes of 32 rows, in phases
    (90, 5, 4, 2048, 4104, "skewed"),
    (300, 2, 2, 5000, 136, "uniform"),   # tiles
    (700, 200, 8, 136, 24, "few"),       # tiles of all rows on few of the experts
    (4100, 5, 4, 264, 1032, "skewed"),   # E2M1: tiles of 128 rows
    (4097, 3, 3, 1032, 1400, "uniform"),
    (1500, 200, 8, 136, 1400, "uniform"),  # as many tiles, but few rows an expert
])
def test_long_and_odd_products_of_integers_are_exact(T, E, k, K, N, kind, fmt, group, dev):
    say(f"[experts4] exact, long T={T} E={E} k={k} K={K} N={N} {kind} {fmt} {group}")
    rng = np.random.default_rng(T)
    idx, off, x, codes, scales, b, _ = inputs(rng, T, E, k, K, N, kind, "swiglu", fmt, group, True)
    plan = routed(idx, E, 1, 8, dev)
    w, _ = block_ref.values4(codes, scales, fmt, group)
    z = np.concatenate([x[off[e]: off[e + 1]] @ w[e].T + b[e] for e in range(E)])
    assert np.abs(z).max() < 2 ** 20
    # plain, the gate and the up projection side by side, then the up projection gated
    w4, xd, bd = packed(codes, scales, fmt, group, dev), bf16(x, dev), torch.from_numpy(b.astype(np.float32)).to(dev)
    assert np.array_equal(f64(plan.expert_linear4(xd, w4, bd)), rounded(z))
    got = f64(plan.expert_linear4(xd, w4, bd, activation="swiglu"))
    want = ref.act("swiglu", z[:, :N]) * z[:, N:]
    # sigmoid's float32 roundings (as for bf16 weights) and one to bf16
    assert (np.abs(got - want) <= (272 * ref.U + ref.BF16_HALF) * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("T", [4, 37, 700])
def test_values_that_are_not_finite_stay_in_their_rows(T, fmt, group, dev):
    rng = np.random.default_rng(T)
    E, k, K, N = 4, 2, 72, 136
    idx, off, x, codes, scales, _, _ = inputs(rng, T, E, k, K, N, "uniform", "none", fmt, group)
    plan = routed(idx, E, 1, 8, dev)
    w4 = packed(codes, scales, fmt, group, dev)
    clean = plan.expert_linear4(bf16(x, dev), w4)
    hit = [off[1], off[2] + (off[3] - off[2]) // 2]
    assert off[1] < off[2] < off[3]
    x[hit[0]], x[hit[1]] = np.nan, np.inf
    got = plan.expert_linear4(bf16(x, dev), w4)
    rows = np.setdiff1d(np.arange(off[-1]), hit)
    assert torch.equal(got[rows], clean[rows]) and not torch.isfinite(got[hit].float()).any()
    # and a scale that is NaN in its weight row
    bad = scales.astype(np.float64).copy()
    bad[2, 5, 0] = 255 if fmt == "e2m1" else np.nan
    x[hit] = 1.0
    clean = plan.expert_linear4(bf16(x, dev), w4)
    got = plan.expert_linear4(bf16(x, dev), packed(codes, bad, fmt, group, dev))
    of_2 = np.arange(off[2], off[3])
    assert torch.isnan(got[of_2, 5].float()).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[of_2, 5] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("fmt,group", [("int4", 64), ("e2m1", 32)])
@pytest.mark.parametrize("T,band,E,k,K,N,act", [(1000, 256, 6, 2, 136, 72, "swiglu"),
                                                (260, 256, 40, 1, 64, 64, "silu"),
                                                (2600, 1280, 3, 2, 264, 520, "none")])
def test_banded_plans(T, band, E, k, K, N, act, fmt, group, dev):
    say(f"[experts4] banded T={T} band={band} E={E} k={k} K={K} N={N} {act} {fmt}")
    rng = np.random.default_rng(T + N)
    idx, _, x, codes, scales, b, _ = inputs(rng, T, E, k, K, N, "uniform", act, fmt, group)
    idx[5, 0] = -1          # a dropped slot: the band's last row stays as it is
    plan = routed(idx, E, 1, 64, dev, band_tokens=band)
    full = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=dev)
    y = plan.expert_linear4(bf16(x, dev), packed(codes, scales, fmt, group, dev),
                            torch.from_numpy(b.astype(np.float32)).to(dev), None, act, y=full)
    for o in plan.read("expert_offsets").reshape(-1, E + 1):
        s = slice(o[0], o[-1])
        want, ey = block_ref.expert_linear4(x[s], codes, scales, fmt, group, b, None, act, o - o[0])
        check(y[s], want, ey, "y")
    assert (y[band * k - 1] == 7).all()


def test_empty_batch(dev):
    w4 = cs.quantize_experts4(torch.ones(5, 40, 64, dtype=torch.bfloat16, device=dev))
    plan = cs.Plan(0, 64, 5, 2, 1).route(torch.empty(0, 2, dtype=torch.int32, device=dev))
    assert plan.expert_linear4(torch.empty(0, 64, dtype=torch.bfloat16, device=dev), w4).shape == (0, 40)


def block(T, H, I, E, k, R, dev, seed, fmt, group, **kw):
    """One decoding block, as it is used: norm, gate, router, shuffle, 4-bit experts, combine, and the
    norm of the block that follows."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rand = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=dev) * scale  # noqa: E731
    p = cs.Plan(T, H, E, k, R, **kw)
    x, delta = rand(T, H).bfloat16(), rand(T, H).bfloat16()
    gamma, gate = 1 + rand(H, scale=0.1), rand(H, E, scale=H ** -0.5)
    w1 = cs.quantize_experts4(rand(E, 2 * I, H, scale=H ** -0.5).bfloat16(), fmt, group)
    w2 = cs.quantize_experts4(rand(E, H, I, scale=I ** -0.5).bfloat16(), fmt, group)
    b1 = rand(E, 2 * I)

    def step():
        h, total, _ = cs.norm(p, x, gamma, residual=delta, kind="rms")
        idx, w = cs.router(p, h.float() @ gate)
        p.route(idx)
        recv, _ = cs.dispatch(p, h)
        mid = cs.expert_linear4(p, recv, w1, b1, activation="swiglu")
        y = cs.expert_linear4(p, mid, w2)
        out = cs.combine(p, y, w)
        after, stream, stats = cs.norm(p, total, gamma, residual=out, kind="rms", save_stats=True)
        return dict(h=h, total=total, idx=idx, w=w, recv=recv, mid=mid, y=y, out=out, after=after,
                    stream=stream, stats=stats)
    return step, dict(p=p, x=x, delta=delta, gamma=gamma, w1=w1, w2=w2, b1=b1)


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("e2m1", 32)])
@pytest.mark.parametrize("T,kw", [(1, {}), (16, {}), (500, dict(ranks_per_node=1, node_dedup=True))])
def test_block_step_by_step(T, kw, fmt, group, dev):
    # Every operator's output against its definition on the GPU's own inputs to it.
    H, I, E, k = 264, 136, 10, 3
    step, m = block(T, H, I, E, k, 5, dev, T, fmt, group, **kw)
    s = step()
    _, off = ref.layout(s["idx"].cpu().numpy(), E)
    norm = block_ref.norm(f64((m["x"].float() + m["delta"].float()).bfloat16()), f64(m["gamma"]), 0.0,
                          True, float(np.float32(1e-5)))["y"]
    check(s["h"], norm[0], block_ref.stored(*norm, "bf16"), "h")

    def product(x, w4, bias, act, got):
        # the definition on the weights' values: codes that stand for them under scales of 1
        w = f64(w4.values())
        z, ez = ref.product(f64(x), w, bias, off)
        K = x.shape[1]
        for e in range(E):
            a = slice(off[e], off[e + 1])
            if fmt == "int4":   # the offset's roundings: scale <= max |w| of the group / 7 * (1 + 2^-8)
                n = -(-K // group)
                full = np.zeros((w.shape[1], n * group))
                full[:, :K] = np.abs(w[e])
                scale = np.repeat(full.reshape(-1, n, group).max(2) / 6.9, group, 1)[:, :K]
                ez[a] += (2 * group + 2) * 2 * ref.U * 279 * (np.abs(f64(x)[a]) @ scale.T)
        if act == "swiglu":
            n = z.shape[1] // 2
            y = ref.act(act, z[:, :n]) * z[:, n:]
            ey = ref.SLOPE * ez[:, :n] * (np.abs(z[:, n:]) + ez[:, n:]) + \
                np.abs(ref.act(act, z[:, :n])) * ez[:, n:] + 272 * ref.U * np.abs(y)
        else:
            y, ey = z, ez
        check(got, y, block_ref.stored(y, ey, "bf16"), act)

    product(s["recv"], m["w1"], f64(m["b1"]), "swiglu", s["mid"])
    product(s["mid"], m["w2"], None, "none", s["y"])
    assert torch.equal(s["stream"], (s["total"].float() + s["out"].float()).bfloat16())
    norm = block_ref.norm(f64(s["stream"]), f64(m["gamma"]), 0.0, True, float(np.float32(1e-5)))["y"]
    check(s["after"], norm[0], block_ref.stored(*norm, "bf16"), "after")


def test_blocks_in_a_graph_and_on_another_stream(dev):
    # Two blocks captured into two graphs, replayed in turn between eager steps of both.
    steps = [block(n, 264, 136, 12, 4, 3, dev, n, f, g)[0] for n, f, g in ((16, "int4", 32), (300, "e2m1", 32))]
    eager = [s() for s in steps]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = steps[0]()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same = lambda a, b: [n for n in a if not torch.equal(a[n], b[n])]  # noqa: E731
    assert same(eager[0], other) == []
    graphs, outs = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s())
        graphs.append(g)
    for i in range(4):
        for j in (0, 1):
            for t in outs[j].values():
                t.zero_()
            graphs[j].replay()
            if i % 2:
                torch.cuda.synchronize()
            assert same(eager[1 - j], steps[1 - j]()) == []
            torch.cuda.synchronize()
            assert same(eager[j], outs[j]) == [], (i, j)


def test_product_captured_on_its_own(dev):
    # The offsets' scan that a small plan leaves to the product is recorded with it: a replay
    # computes with the plan's latest route.
    rng = np.random.default_rng(2)
    T, E, k, K, N = 90, 7, 2, 72, 136
    idx, _, x, codes, scales, _, _ = inputs(rng, T, E, k, K, N, "uniform", "none", "int4", 32)
    routes = [torch.from_numpy(i).to(dev) for i in (idx, random_routing(rng, T, E, k, "skewed"))]
    xd, w4 = bf16(x, dev), packed(codes, scales, "int4", 32, dev)
    want = [cs.Plan(T, 8, E, k, 1).route(i).expert_linear4(xd, w4) for i in routes]
    assert not torch.equal(*want)
    plan = cs.Plan(T, 8, E, k, 1).route(routes[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = plan.expert_linear4(xd, w4)
    assert torch.equal(plan.expert_linear4(xd, w4), want[0])
    for i in (0, 1, 0, 1):
        plan.route(routes[i])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(plan.expert_linear4(xd, w4), want[i])


def test_given_stream_and_output(dev):
    step, m = block(40, 72, 64, 6, 2, 1, dev, 4, "int4", 64)
    s = step()
    side = torch.cuda.Stream()
    late = torch.zeros_like(s["recv"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(50):
            late.add_(1)
        late.copy_(s["recv"])
    y = torch.empty_like(s["mid"])
    got = cs.expert_linear4(m["p"], late, m["w1"], m["b1"], activation="swiglu", y=y, stream=side)
    values = m["w1"].values(stream=side)
    side.synchronize()
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, s["mid"])
    assert torch.equal(values, m["w1"].values())
    square = cs.quantize_experts4(torch.ones(6, 72, 72, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError, match="shares"):
        m["p"].expert_linear4(s["recv"], square, y=s["recv"])


def test_timing_names_every_launch(dev):
    names = set()
    for T in (4, 300, 4000):
        step, m = block(T, 264, 136, 12, 4, 3, dev, 5, "int4", 128)
        m["p"].timing(64)
        step()
        names |= {n for n, _, ms in m["p"].timing_read() if ms > 0}
        m["p"].timing(0)
    assert {_abi.kernel_name(i) for i in _abi.BLOCK_KERNELS} <= names | {"norm_grad_kernel", "norm_sum_kernel"}


@pytest.mark.slow
@pytest.mark.parametrize("fmt,group", [("int4", 128), ("e2m1", 32)])
def test_offsets_past_32_bits(fmt, group, dev):
    # Rows whose bytes pass 2^32, and packed weights past 2^32 bytes: the last rows, of the last expert.
    T, k, E, H, N = 70000, 8, 16, 4096, 8
    rng = np.random.default_rng(0)
    plan = routed(random_routing(rng, T, E, k), E, 1, H, dev)
    assert T * k * H > 2 ** 31
    x = torch.randint(-2, 3, (T * k, H), device=dev).bfloat16()
    codes, scales = draw(rng, E, N, H, fmt, group, True)
    w4 = packed(codes, scales, fmt, group, dev)
    y = plan.expert_linear4(x, w4)
    tail = slice(T * k - 500, T * k)
    assert plan.read("expert_offsets")[E - 1] < T * k - 500
    assert torch.equal(y[tail].double(), (x[tail].double() @ w4.values()[E - 1].double().t()).bfloat16().double())
    del x, y, w4
    E, Z, K = 300, 8192, 4096
    codes = torch.randint(0, 256, (E, Z, K // 2), dtype=torch.uint8, device=dev)
    s = torch.full((E, Z, K // group), 127, dtype=torch.uint8, device=dev)
    s = s if fmt == "e2m1" else torch.ones_like(s, dtype=torch.bfloat16)
    w4 = cs.pack_experts4(codes, s, fmt, group)
    assert w4.packed.numel() > 2 ** 32
    plan = cs.Plan(3, 8, E, 1, 1).route(torch.full((3, 1), E - 1, dtype=torch.int32, device=dev))
    x = torch.randint(-1, 2, (3, K), device=dev).bfloat16()
    c = codes[E - 1].long()
    c = torch.stack([c & 15, c >> 4], 2).reshape(Z, K)
    table = torch.tensor(block_ref.INT4 if fmt == "int4" else block_ref.E2M1, device=dev)
    want = x.double() @ table[c].t().contiguous()
    assert torch.equal(plan.expert_linear4(x, w4).double(), want.bfloat16().double())
    del codes, w4, c
    torch.cuda.empty_cache()
