"""E2M1 products at the ends of E8M0's range: scales of 2^-127 to 2^-125, under which weights are
subnormal in bf16, and of 2^125 to 2^127, under which some are past its range and stand for infinities."""

import numpy as np
import pytest
import torch

import layer_ref as ref
from block_ref import E2M1

from gpu_util import say
from test_gpu_experts4 import packed
from test_gpu_layer import bf16, f64, random_routing, rounded, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


SIZES = [  # T, E, k, K, N: passes of 16 and of 32 rows, tiles of 64 and of 128 rows
    (1, 6, 2, 264, 40), (16, 16, 4, 136, 72), (40, 2, 2, 392, 136), (600, 3, 2, 264, 520),
    (4100, 5, 4, 136, 2064),
]


def products(T, E, k, K, N, bytes_, power, dev, rng, codes):
    """(result, the products' operands): x is +-1 to +-3 times 2^power."""
    idx = random_routing(rng, T, E, k)
    _, off = ref.layout(idx, E)
    scales = rng.choice(bytes_, size=(E, N, -(-K // 32)))
    x = rng.integers(1, 4, size=(T * k, K)) * rng.choice([-1, 1], size=(T * k, 1))
    plan = routed(idx, E, 1, 8, dev)
    got = plan.expert_linear4(bf16(np.ldexp(x.astype(float), power), dev),
                              packed(codes, scales, "e2m1", 32, dev))
    return f64(got), x.astype(float), scales, off


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
@pytest.mark.parametrize("bytes_,power", [((0, 1, 2), 122), ((252,), -126), ((250, 251, 252), -126)])
def test_products_under_extreme_scales_are_exact(T, E, k, K, N, bytes_, power, dev):
    say(f"[experts4] scales {bytes_} T={T} E={E} k={k} K={K} N={N}")
    rng = np.random.default_rng(T + K)
    codes = rng.integers(0, 16, size=(E, N, K))
    got, x, scales, off = products(T, E, k, K, N, bytes_, power, dev, rng, codes)
    # halves times integers, relative to the smallest scale
    w = E2M1[codes] * np.repeat(np.ldexp(1.0, scales - min(bytes_)), 32, 2)[:, :, :K]
    z = np.concatenate([x[off[e]: off[e + 1]] @ w[e].T for e in range(E)])
    assert np.abs(z).max() < 2 ** 22
    assert np.array_equal(got, rounded(np.ldexp(z, min(bytes_) - 127 + power)))


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
@pytest.mark.parametrize("byte", [253, 254])
def test_weights_past_the_range_are_infinite(T, E, k, K, N, byte, dev):
    # Infinite from 4 * 2^126 and from 2 * 2^127 on.  x is nowhere 0 and of one sign in a row, so a
    # result is infinite, or NaN where infinite weights of both signs meet.
    say(f"[experts4] scale {byte} T={T} E={E} k={k} K={K} N={N}")
    rng = np.random.default_rng(T + K)
    limit = 4 if byte == 253 else 2
    within = np.flatnonzero(np.abs(E2M1) < limit)
    codes = within[rng.integers(0, within.size, size=(E, N, K))]
    past = np.flatnonzero(E2M1 >= limit)
    codes[:, 1, K // 2] = past[rng.integers(past.size)]
    codes[:, 2, K - 1] = past[-1] + 8
    codes[:, 3, 0], codes[:, 3, 40] = past[0], past[0] + 8
    got, x, scales, off = products(T, E, k, K, N, (byte,), -126, dev, rng, codes)
    w = E2M1[codes]
    z = np.concatenate([x[off[e]: off[e + 1]] @ w[e].T for e in range(E)])
    want = rounded(np.ldexp(z, byte - 127 - 126))
    sign = x[:, 0]
    want[:, 1], want[:, 2], want[:, 3] = sign * np.inf, -sign * np.inf, np.nan
    assert np.array_equal(got, want, equal_nan=True)
