"""INT4 products: a group's sum of x * (code - 8) is taken as one of x * (16 + code) and of x * -24,
so that integers below 2^24 / 24 in magnitude add up without a rounding, and x below 2^116 without an
overflow.  Whatever the order, a partial sum of a group is at most 24 times the magnitudes' sum."""

import numpy as np
import pytest
import torch

import block_ref
import layer_ref as ref

from gpu_util import say
from test_gpu_experts4 import packed
from test_gpu_layer import bf16, f64, random_routing, rounded, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


SIZES = [  # T, E, k, K, N: passes of 16 and of 32 rows, tiles of few and of many rows
    (1, 6, 2, 520, 40), (16, 16, 4, 1000, 72), (40, 2, 2, 512, 136), (280, 140, 6, 264, 72),
    (900, 5, 2, 264, 264),
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_large_x_of_weight_zero_takes_nothing_from_the_others(T, E, k, K, N, group, dev):
    # The last x of each whole group is +-255 * 2^9, and its weights are 0 (code 8); of the others 24 a
    # row are +-1.  Exact results are integers up to 24 * 8, which bf16 holds, and no partial sum of a
    # group passes 24 * (255 * 2^9 + 24) < 2^22.
    say(f"[experts4] sums T={T} E={E} k={k} K={K} N={N} int4 {group}")
    rng = np.random.default_rng(T + K + group)
    idx = random_routing(rng, T, E, k)
    _, off = ref.layout(idx, E)
    large = np.arange(group - 1, K // group * group, group)
    assert large.size
    codes = rng.integers(0, 16, size=(E, 2 * N, K))
    codes[:, :, large] = 8
    scales = np.ones((E, 2 * N, -(-K // group)))
    x = np.zeros((T * k, K))
    small = np.setdiff1d(np.arange(K), large)
    for r in range(T * k):
        x[r, rng.choice(small, 24, replace=False)] = rng.choice([-1, 1], 24)
    x[:, large] = rng.choice([-255 * 2 ** 9, 255 * 2 ** 9], size=(T * k, large.size))
    plan, w4 = routed(idx, E, 1, 8, dev), packed(codes, scales, "int4", group, dev)
    z = np.concatenate([x[off[e]: off[e + 1]] @ (codes[e] - 8.0).T for e in range(E)])
    assert np.abs(z).max() <= 24 * 8
    xd = bf16(x, dev)
    assert np.array_equal(f64(plan.expert_linear4(xd, w4)), z)
    got = f64(plan.expert_linear4(xd, w4, activation="swiglu"))
    want = ref.act("swiglu", z[:, :N]) * z[:, N:]
    # sigmoid's float32 roundings (as for bf16 weights) and one to bf16
    assert (np.abs(got - want) <= (272 * ref.U + ref.BF16_HALF) * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_x_just_below_the_limit(T, E, k, K, N, group, dev):
    # x of magnitude 255 * 2^108, just below 2^116, everywhere: 24 * 128 of them are 2^127.6.  Under scales
    # of 2^-110 results are integers times 255 / 4, exact in float32.
    say(f"[experts4] limit T={T} E={E} k={k} K={K} N={N} int4 {group}")
    rng = np.random.default_rng(T + K + group)
    idx = random_routing(rng, T, E, k)
    _, off = ref.layout(idx, E)
    codes = rng.integers(0, 16, size=(E, N, K))
    scales = np.full((E, N, -(-K // group)), 2.0 ** -110)
    sign = np.repeat(rng.choice([-1.0, 1.0], size=(T * k, -(-K // 8))), 8, 1)[:, :K]
    sign[::3] = 1.0                                  # the largest sums of one sign
    plan, w4 = routed(idx, E, 1, 8, dev), packed(codes, scales, "int4", group, dev)
    got = plan.expert_linear4(bf16(sign * (255 * 2.0 ** 108), dev), w4)
    z = np.concatenate([sign[off[e]: off[e + 1]] @ (codes[e] - 8.0).T for e in range(E)])
    assert np.abs(z).max() * 255 < 2 ** 24
    assert np.array_equal(f64(got), rounded(z * (255 / 4)))


def test_packed_words_hold_every_code(dev):
    # Each code at each of a word's eight places, in every group size, through the values and a product
    # with the unit vectors.
    K = 128
    codes = (np.arange(16)[:, None] + np.arange(K)[None, :] * 5) % 16
    codes = codes[None].astype(int)
    for group in (32, 64, 128):
        scales = np.ones((1, 16, K // group))
        w4 = packed(codes, scales, "int4", group, dev)
        want, _ = block_ref.values4(codes, scales, "int4", group)
        assert np.array_equal(f64(w4.values()), want)
        plan = routed(np.zeros((K, 1), dtype=np.int32), 1, 1, 8, dev)
        assert np.array_equal(f64(plan.expert_linear4(bf16(np.eye(K), dev), w4)), want[0].T)
