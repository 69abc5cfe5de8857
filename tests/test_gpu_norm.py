"""The norm of the residual stream and its gradient on the GPU against their float64 definitions
(block_ref.py): every output element within the bound derived there."""

import numpy as np
import pytest
import torch

import block_ref as ref
import combine_shuffling_amd as cs
from combine_shuffling_amd import _abi

from gpu_util import say

pytestmark = pytest.mark.gpu

U = ref.U
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def tensor(a, dtype, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TYPES[dtype]).to(dev)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} elements outside; at {i}: {got[i]!r}, "
                             f"want {want[i]!r} +- {np.broadcast_to(bound, got.shape)[i]!r}")


def plan(T, H, **kw):
    return cs.Plan(T, H, 4, 1, 2, **kw)


SIZES = [  # T, H: a row in 16 or 32 lanes, a wave, 2 to 16 waves, two chunks a lane; one and many turns
    (1, 8), (3, 24), (5, 128), (130, 136), (257, 256), (61, 512), (40, 520), (33, 1000), (300, 2048),
    (20, 4096), (9, 7168), (17, 8192), (5, 8200), (3, 16384), (4099, 264), (40000, 8), (700, 5000),
]


def stream(rng, T, H, dtype, dev):
    """Rows with a few wide columns and their own means, and their float64 values."""
    x = rng.normal(size=(T, H)) * np.where(rng.random(H) < 0.03, 30.0, 1.0) + 2 * rng.normal(size=(T, 1))
    t = tensor(x, dtype, dev)
    return t, f64(t)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_norm(T, H, xt, yt, dev):
    say(f"[norm] forward T={T} H={H} {xt} -> {yt}")
    rng = np.random.default_rng(T + H)
    p = plan(T, H)
    x, xv = stream(rng, T, H, xt, dev)
    r, _ = stream(rng, T, H, xt, dev)
    gamma, beta = tensor(rng.normal(size=H), "f32", dev), tensor(rng.normal(size=H), "f32", dev)
    sum_ = (x.float() + r.float()).to(x.dtype)
    for kind in ("layer", "rms"):
        for res in (None, r):
            for g, b in ((gamma, beta), (gamma, None), (None, None)):
                full = torch.full((T + 1, H), 7.0, dtype=TYPES[yt], device=dev)
                y, total, stats = p.norm(x, g, b, res, kind, 1e-5, TYPES[yt], save_stats=True, y=full[:T])
                assert (full[T] == 7).all()
                if res is None:
                    assert total is None
                else:
                    assert torch.equal(total, sum_)
                want = ref.norm(xv if res is None else f64(sum_), 1.0 if g is None else f64(g),
                                0.0 if b is None else f64(b), kind == "rms", np.float64(np.float32(1e-5)))
                what = f"{kind} residual {res is not None}"
                check(stats[:, 0], *want["mean"], f"mean {what}")
                check(stats[:, 1], *want["rstd"], f"rstd {what}")
                v, e = want["y"]
                check(y, v, ref.stored(v, e, yt), f"y {what}")
    again = p.norm(x, gamma, beta, r, "rms", out_dtype=TYPES[yt])
    assert again[2] is None
    assert torch.equal(again[0], p.norm(x, gamma, beta, r, "rms", out_dtype=TYPES[yt], save_stats=True)[0])


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("gt", ["bf16", "f32"])
def test_norm_backward(T, H, xt, gt, dev):
    say(f"[norm] backward T={T} H={H} {xt}, gradient {gt}")
    rng = np.random.default_rng(T + 2 * H)
    p = plan(T, H)
    x, xv = stream(rng, T, H, xt, dev)
    gy, gv = tensor(rng.normal(size=(T, H)), gt, dev), None
    gv = f64(gy)
    join = tensor(rng.normal(size=(T, H)), xt, dev)
    gamma = tensor(rng.normal(size=H), "f32", dev)
    for kind in ("layer", "rms"):
        r = ref.norm(xv, 1.0, 0.0, kind == "rms", 1e-5)
        stats = tensor(np.stack([r["mean"][0], r["rstd"][0]], 1), "f32", dev)
        for g, j in ((gamma, None), (gamma, join), (None, None)):
            full = torch.full((T + 1, H), 7.0, dtype=TYPES[xt], device=dev)
            gx, gg, gb = p.norm_backward(gy, x, stats, g, j, kind, grad_x=full[:T])
            assert (full[T] == 7).all()
            want = ref.norm_backward(gv, xv, f64(stats), 1.0 if g is None else f64(g),
                                     None if j is None else f64(j), kind == "rms")
            v, e = want["grad_x"]
            check(gx, v, ref.stored(v, e, xt), f"grad_x {kind}")
            check(gg, *want["grad_gamma"], f"grad_gamma {kind}")
            check(gb, *want["grad_beta"], f"grad_beta {kind}")
        # one at a time, the same bits
        every = p.norm_backward(gy, x, stats, gamma, join, kind)
        for i in range(3):
            one = p.norm_backward(gy, x, stats, gamma, join, kind, i == 0, i == 1, i == 2)
            assert [t is not None for t in one] == [q == i for q in range(3)]
            assert torch.equal(one[i], every[i])


def test_sums_of_integers_are_exact(dev):
    # mean 0 and rstd 1 given, small integers: the weights' gradients are exact whatever the order.
    rng = np.random.default_rng(1)
    for T, H in ((3, 24), (1000, 40), (2000, 1024), (5000, 264), (600, 7168)):
        x, gy = rng.integers(-2, 3, size=(T, H)), rng.integers(-2, 3, size=(T, H))
        stats = torch.tensor([0.0, 1.0], device=dev).repeat(T, 1)
        _, gg, gb = plan(T, H).norm_backward(tensor(gy, "bf16", dev), tensor(x, "bf16", dev), stats)
        assert np.array_equal(f64(gg), (gy * x).sum(0)) and np.array_equal(f64(gb), gy.sum(0))


def test_no_rows(dev):
    p = cs.Plan(0, 64, 4, 1, 2)
    x = torch.empty(0, 64, device=dev)
    y, total, stats = p.norm(x, residual=x.clone(), save_stats=True)
    assert y.shape == total.shape == (0, 64) and stats.shape == (0, 2)
    gx, gg, gb = p.norm_backward(y, x, stats, grad_gamma=torch.full((64,), 7.0, device=dev))
    assert gx.shape == (0, 64) and not gg.any() and not gb.any()


@pytest.mark.parametrize("H", [40, 1000, 2056, 16384])
def test_values_that_are_not_finite_stay_in_their_rows(H, dev):
    T = 37
    rng = np.random.default_rng(H)
    p = plan(T, H)
    x, _ = stream(rng, T, H, "f32", dev)
    gy = tensor(rng.normal(size=(T, H)), "bf16", dev)
    y, _, stats = p.norm(x, save_stats=True)
    gx, _, gb = p.norm_backward(gy, x, stats)
    bad, worse = x.clone(), gy.clone()
    bad[3, H // 2], bad[11, 0] = float("nan"), float("inf")
    worse[20, 1] = float("nan")
    y2, _, stats2 = p.norm(bad, save_stats=True)
    gx2, _, gb2 = p.norm_backward(worse, bad, stats2)
    rows = [r for r in range(T) if r not in (3, 11)]
    assert torch.equal(y[rows], y2[rows]) and torch.equal(stats[rows], stats2[rows])
    assert torch.isnan(y2[3]).all() and torch.isnan(y2[11]).all()
    rows.remove(20)
    assert torch.equal(gx[rows], gx2[rows]) and torch.isnan(gx2[[3, 11, 20]]).all()
    assert torch.isnan(gb2[1]) and torch.equal(gb[2:], gb2[2:])


def test_constant_zero_and_huge_rows(dev):
    H = 264
    p = plan(4, H)
    x = torch.zeros(4, H, device=dev)
    x[1], x[2], x[3] = 5.0, 1e30, torch.linspace(-1, 1, H, device=dev) * 1e18
    for kind in ("layer", "rms"):
        y, _, stats = p.norm(x, kind=kind, out_dtype=torch.float32, save_stats=True)
        assert (y[0] == 0).all()
        assert abs(stats[0, 1].item() * 1e-5 ** 0.5 - 1) < 1e-6
        want = ref.norm(f64(x), 1.0, 0.0, kind == "rms", float(np.float32(1e-5)))
        for r in ((0, 1, 3) if kind == "layer" else (0, 3)):
            assert (np.abs(f64(y)[r] - want["y"][0][r]) <= want["y"][1][r] + 2.0 ** -120).all(), (kind, r)
        if kind == "rms":       # squares past float32's range: rstd 0
            assert stats[2, 1] == 0 and (y[2] == 0).all()
    y, _, _ = p.norm(x, eps=0.0, out_dtype=torch.float32)
    assert torch.isnan(y[0]).all()              # 0 / 0, as the formula


def test_given_stream_outputs_and_workspace(dev):
    rng = np.random.default_rng(0)
    T, H = 3000, 520
    p = plan(T, H)
    x, _ = stream(rng, T, H, "bf16", dev)
    gamma = tensor(rng.normal(size=H), "f32", dev)
    want = p.norm(x, gamma, residual=x.clone(), save_stats=True)
    back = p.norm_backward(x, want[1], want[2], gamma)
    side = torch.cuda.Stream()
    late = torch.zeros_like(x)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(50):
            late.add_(1)
        late.copy_(x)
    outs = [torch.empty_like(t) for t in want]
    got = cs.norm(p, late, gamma, None, x, y=outs[0], total=outs[1],
                  stats=outs[2], stream=side)
    given = [torch.empty_like(t) for t in back]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=dev)
    again = cs.norm_backward(p, late, outs[1], outs[2], gamma, grad_x=given[0], grad_gamma=given[1],
                             grad_beta=given[2], workspace=ws, stream=side)
    side.synchronize()
    for o, g, w in zip(outs + given, got + again, want + back):
        assert o.data_ptr() == g.data_ptr() and torch.equal(o, w)
    with pytest.raises(cs.MoeError):      # a workspace that is not 256-byte aligned
        cs.norm_backward(p, x, want[1], want[2], gamma, workspace=ws[16:])
    with pytest.raises(ValueError, match="shares"):
        cs.norm_backward(p, x, want[1], want[2], gamma, grad_x=want[1])


def test_captured_and_replayed(dev):
    # Two steps in one graph, on plans that share nothing, between eager calls on the same plans.
    rng = np.random.default_rng(5)
    plans = [plan(900, 1000), plan(2, 7168)]
    data = []
    for p in plans:
        x, _ = stream(rng, p.T, p.H, "f32", dev)
        data.append((x, x.clone().mul_(0.5), tensor(rng.normal(size=p.H), "f32", dev),
                     tensor(rng.normal(size=(p.T, p.H)), "bf16", dev)))

    def step(i):
        x, r, gamma, gy = data[i]
        y, total, stats = plans[i].norm(x, gamma, gamma, r, save_stats=True)
        return (y, total, stats, *plans[i].norm_backward(gy, total, stats, gamma, r))

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [step(0), step(1)]
    for n in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        graph.replay()
        if n % 2:
            torch.cuda.synchronize()
        eager = [step(0), step(1)]
        torch.cuda.synchronize()
        for i in range(2):
            for a, b, c in zip(want[i], outs[i], eager[i]):
                assert torch.equal(a, b) and torch.equal(a, c)


def test_timing_names_the_kernels(dev):
    p = plan(3000, 64)
    p.timing(8)
    x = torch.randn(3000, 64, device=dev)
    _, _, stats = p.norm(x, save_stats=True)
    p.norm_backward(x.bfloat16(), x, stats)
    names = [n for n, _, ms in p.timing_read() if ms > 0]
    assert names == [_abi.kernel_name(i) for i in _abi.BLOCK_KERNELS][:3]


@pytest.mark.slow
def test_offsets_past_32_bits(dev):
    T, H = 300000, 8192
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    x = torch.randint(-3, 4, (T, H), generator=g, device=dev, dtype=torch.int8).to(torch.bfloat16)
    p = plan(T, H)
    assert x.numel() > 2 ** 31
    y, total, stats = p.norm(x, residual=x, kind="rms", eps=0.0, save_stats=True)
    tail = slice(T - 300, T)
    assert torch.equal(total[tail], 2 * x[tail])
    few = plan(300, H)
    want = few.norm(x[tail].contiguous(), residual=x[tail].clone(), kind="rms", eps=0.0, save_stats=True)
    assert torch.equal(want[0], y[tail]) and torch.equal(want[2], stats[tail])
    del y
    one = torch.tensor([0.0, 1.0], device=dev).repeat(T, 1)
    gx, gg, gb = p.norm_backward(x, total, one, kind="rms")
    wx, _, _ = few.norm_backward(x[tail].contiguous(), total[tail].contiguous(), one[tail], kind="rms")
    assert torch.equal(gx[tail], wx)
    part = 30000
    sums = sum((x[a: a + part].double() ** 2).sum(0) for a in range(0, T, part))
    assert torch.equal(gg.double(), 2 * sums)          # integers below 2^24
    assert torch.equal(gb.double(), sum(x[a: a + part].double().sum(0) for a in range(0, T, part)))
    del x, total, gx
    torch.cuda.empty_cache()
