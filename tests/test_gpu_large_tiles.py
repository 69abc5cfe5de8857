"""The experts' gradients where their large tiles (256 x 256) are taken, with many and uneven rows an
expert: none, a few, tiles filled in part, several tiles; and nodes of more than 256 experts."""

import math

import pytest
import torch

import combine_shuffling_amd as cs
import layer_ref as ref
import test_gpu_layer as layer

from gpu_util import say

pytestmark = pytest.mark.gpu

U = ref.U
E, K = 64, 776
# 64 * ceil(1032 / 256) * ceil(776 / 256) = 1280 weight tiles: at least four a CU
ROWS = [0, 1, 5, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300, 384, 511,
        513, 700, 0, 0, 17, 2, 321, 64, 8, 0]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def uneven(dev, seed):
    """A plan of one expert a token, and the experts' first rows."""
    g = torch.Generator().manual_seed(seed)
    rows = torch.tensor(ROWS + [(7 * n) % 90 for n in ROWS])
    ids = torch.repeat_interleave(torch.arange(E), rows)
    ids = ids[torch.randperm(len(ids), generator=g)]
    plan = cs.Plan(len(ids), 8, E, 1, 1).route(ids.int()[:, None].contiguous().to(dev))
    off = [0, *torch.cumsum(rows, 0).tolist()]
    assert plan.read("expert_offsets").tolist() == off
    return plan, off


def by_expert(off):
    return [(e, slice(off[e], off[e + 1])) for e in range(E)]


def test_integers_are_exact(dev):
    say("[large tiles] integers")
    plan, off = uneven(dev, 0)
    g = torch.Generator(device=dev).manual_seed(1)
    Z = 1032
    draw = lambda *s: torch.randint(-2, 3, s, generator=g, device=dev).bfloat16()  # noqa: E731
    x, w, gy = draw(off[-1], K), draw(E, Z, K), draw(off[-1], Z)
    y, _ = plan.expert_linear(x, w)
    gx, gw, gb = plan.expert_linear_backward(gy, x, w, bias_grad=True, grad_w_dtype=torch.float32)
    alone = [plan.expert_linear_backward(gy, x, w, x_grad=i == 0, w_grad=i == 1, bias_grad=i == 2,
                                         grad_w_dtype=torch.float32)[i] for i in range(3)]
    half = plan.expert_linear_backward(gy, x, w)[1]
    for e, s in by_expert(off):
        a, b, c = x[s].double(), gy[s].double(), w[e].double()
        assert torch.equal(y[s].double(), (a @ c.t().contiguous()).bfloat16().double()), e
        assert torch.equal(gx[s].double(), (b @ c).bfloat16().double()), e
        want = b.t().contiguous() @ a
        assert torch.equal(gw[e].double(), want), e
        assert torch.equal(half[e].double(), want.bfloat16().double()), e
        assert torch.equal(gb[e].double(), b.sum(0)), e
    for one, both in zip(alone, (gx, gw, gb)):
        assert torch.equal(one, both)


@pytest.mark.parametrize("act,N", [("gelu", 1032), ("swiglu", 520)])
def test_gradient_with_activation(act, N, dev):
    # The definition and the bounds of layer_ref.expert_linear_backward, expert by expert in float64.
    say(f"[large tiles] {act}")
    plan, off = uneven(dev, 2)
    g = torch.Generator(device=dev).manual_seed(3)
    Z = 2 * N if act == "swiglu" else N
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, gy, pre = rand(off[-1], K).bfloat16(), rand(off[-1], N).bfloat16(), rand(off[-1], Z).bfloat16()
    w = (rand(E, Z, K) / math.sqrt(K)).bfloat16()
    results = {t: plan.expert_linear_backward(gy, x, w, pre, act, bias_grad=True, grad_w_dtype=t)
               for t in (torch.float32, torch.bfloat16)}

    def inside(got, want, bound, what):
        assert ((got.double() - want).abs() <= bound).all(), what

    half = lambda v, b: b + ref.BF16_HALF * (v.abs() + b) + ref.TINY  # noqa: E731
    for e, s in by_expert(off):
        z, d = pre[s].double(), gy[s].double()
        if act == "swiglu":
            gate, up = z[:, :N], z[:, N:]
            sig = torch.sigmoid(gate)
            gz = torch.cat([d * up * (sig + gate * sig * (1 - sig)), d * gate * sig], 1)
            size = torch.cat([(d * up).abs() * (1 + gate.abs()), (d * gate).abs()], 1)
        else:
            gz = d * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            size = d.abs() * (1 + z.abs())
        ez = 64 * U * size
        eb = half(gz, ez)
        a, c, n = x[s].double(), w[e].double(), off[e + 1] - off[e]
        gx, gw = gz @ c, gz.t().contiguous() @ a
        mag = gz.abs() + eb
        ex = eb @ c.abs() + (Z + 1) * 2 * U * (mag @ c.abs())
        ew = eb.t().contiguous() @ a.abs() + (n + 1) * 2 * U * (mag.t().contiguous() @ a.abs())
        eg = ez.sum(0) + (n + 1) * U * (gz.abs() + ez).sum(0)
        for t, (got_x, got_w, got_b) in results.items():
            inside(got_x[s], gx, half(gx, ex), (e, "grad_x"))
            inside(got_w[e], gw, ew if t == torch.float32 else half(gw, ew), (e, "grad_w", t))
            inside(got_b[e], gz.sum(0), eg, (e, "grad_bias"))


@pytest.mark.parametrize("T,E,k,R,nodes", [(40, 300, 16, 6, 2), (9, 1024, 16, 64, 9), (33, 1000, 11, 7, 3),
                                           (4200, 512, 8, 16, 4), (21, 513, 3, 57, 5)])
@pytest.mark.parametrize("how", ["plain", "bias", "masked", "huge"])
def test_router_nodes_of_many_experts(T, E, k, R, nodes, how, dev):
    layer.test_router(T, E, k, R, 1, nodes, torch.float32, how, dev)
