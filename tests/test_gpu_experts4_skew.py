"""4-bit experts under skewed routing: a busy expert's rows take several passes of the kernel for few
rows, each over a contraction in phases."""

import numpy as np
import pytest
import torch

import block_ref
import layer_ref as ref

from gpu_util import say
from test_gpu_experts4 import FORMATS, IDS, inputs, packed
from test_gpu_layer import bf16, f64, rounded, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("fmt,group", FORMATS, ids=IDS)
@pytest.mark.parametrize("T,E,k,K,N", [
    (48, 40, 2, 5000, 72),      # passes of 16 rows, three phases
    (5, 12, 2, 7168, 40),       # of 8 rows, two phases
    (17, 24, 1, 2056, 136),     # of 16 rows, one row in the second; two phases
    (300, 200, 2, 4104, 24),
])
def test_busy_experts_are_exact(T, E, k, K, N, fmt, group, dev):
    # The first expert has every token, the others share the rest.
    say(f"[experts4] busy T={T} E={E} k={k} K={K} N={N} {fmt} {group}")
    rng = np.random.default_rng(T + K)
    _, _, x, codes, scales, b, _ = inputs(rng, T, E, k, K, N, "uniform", "swiglu", fmt, group, True)
    idx = np.argsort(rng.random((T, E)) - 2.0 * (np.arange(E) == 0), axis=1)[:, :k].astype(np.int32)
    _, off = ref.layout(idx, E)
    assert off[1] == T
    plan = routed(idx, E, 1, 8, dev)
    w, _ = block_ref.values4(codes, scales, fmt, group)
    z = np.concatenate([x[off[e]: off[e + 1]] @ w[e].T + b[e] for e in range(E)])
    assert np.abs(z).max() < 2 ** 20
    w4, xd, bd = packed(codes, scales, fmt, group, dev), bf16(x, dev), torch.from_numpy(b.astype(np.float32)).to(dev)
    assert np.array_equal(f64(plan.expert_linear4(xd, w4, bd)), rounded(z))
    got = f64(plan.expert_linear4(xd, w4, bd, activation="swiglu"))
    want = ref.act("swiglu", z[:, :N]) * z[:, N:]
    # sigmoid's float32 roundings (as for bf16 weights) and one to bf16
    assert (np.abs(got - want) <= (272 * ref.U + ref.BF16_HALF) * np.abs(want) + 1e-30).all()
