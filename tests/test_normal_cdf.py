"""The normal distribution of the experts' GELU: its polynomial in double precision (CPU), and
z * Phi(z) as the kernels compute it in float32."""

import math
import os
import re

import numpy as np
import pytest
import torch

import combine_shuffling_amd as cs

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "combine_shuffling_amd", "csrc", "expert.hip")
U = 2.0 ** -24


def polynomial():
    text = open(SOURCE).read()
    body = text[text.index("float normal_cdf("):]
    body = body[: body.index("return")]
    c = re.findall(r"float p = ([-0-9.]+)f;|fmaf\(p, t, ([-0-9.]+)f\)", body)
    return [float(np.float32(a or b)) for a, b in c]


def test_polynomial():
    c = polynomial()
    assert len(c) == 8
    worst = 0.0
    for z in np.linspace(0.0, 15.0, 30001):
        x = z / math.sqrt(2.0)
        t = 1.0 / (1.0 + 0.425 * x)
        p = 0.0
        for a in c:
            p = p * t + a
        exact = math.erfc(x) * math.exp(x * x)   # both relative to 2^-52 times x^2 at worst
        worst = max(worst, abs(t * p / exact - 1.0))
    assert 1e-7 < worst < 2.2e-7


@pytest.mark.gpu
def test_gelu_in_float32():
    # The bias gradient of an expert's only row is grad_y * gelu(gate), in float32 (GEGLU's up
    # half).  Every bf16 gate from -16 to 16.  Roundings, in 2^-24: exp's argument z^2 (its product
    # with log2 e and that constant's own), its result 2; t 4 and their effect on t P(t) at most
    # 2.65-fold, 11; P's coefficients and steps 7; the fit 3.5; products 4.
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    bits = torch.arange(0, 0x4180 + 1, dtype=torch.int32)
    z = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(torch.bfloat16)
    n = (len(z) + 7) // 8 * 8
    z = torch.cat([z, torch.zeros(n - len(z), dtype=torch.bfloat16)]).to(dev)
    plan = cs.Plan(1, 8, 1, 1, 1).route(torch.zeros(1, 1, dtype=torch.int32, device=dev))
    one = torch.ones(1, n, dtype=torch.bfloat16, device=dev)
    pre = torch.cat([z, one[0]])[None].contiguous()
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(1, 2 * n, 8, dtype=torch.bfloat16, device=dev)
    _, _, gb = plan.expert_linear_backward(one, x, w, pre, "geglu", bias_grad=True, x_grad=False,
                                           w_grad=False)
    got = gb[0, n:].cpu().double().numpy()
    v = z.cpu().double().numpy()
    want = np.array([a * 0.5 * math.erfc(-a / math.sqrt(2.0)) for a in v])
    err = np.abs(got - want)
    tail = v < -12.9
    rel = (v * v + 32) * U
    assert (err[~tail] <= (rel * np.abs(want) + 2.0 ** -126)[~tail]).all()
    assert (err[tail] <= np.abs(v[tail]) * 2.0 ** -125).all()
    used = (np.abs(want) > 2.0 ** -120) & ~tail
    r = err[used] / (np.abs(want[used]) * U)
    print(f"largest relative error {r.max():.1f} x 2^-24 at z = {v[used][r.argmax()]}; "
          f"|z| < 1: {r[np.abs(v[used]) < 1].max():.1f}")
