"""Gradients of the experts' product asked for without the rows that only the others read."""

import pytest
import torch

import combine_shuffling_amd as cs

BF = dict(dtype=torch.bfloat16)


def test_rows_are_needed_for_the_weight_gradient_only():
    p = cs.Plan(64, 64, 8, 2, 2)
    p.device = torch.device("cpu")   # as if routed: the checks come before any launch
    gy, w = torch.zeros(128, 32, **BF), torch.zeros(8, 32, 64, **BF)
    for how in (dict(w_grad=False), dict(w_grad=False, x_grad=False, bias_grad=True)):
        with pytest.raises(ValueError, match="GPU"):     # past every other check
            p.expert_linear_backward(gy, None, w, **how)
    with pytest.raises(TypeError, match="x must be"):
        p.expert_linear_backward(gy, None, w)
    with pytest.raises(ValueError, match="x has shape"):
        p.expert_linear_backward(gy, torch.zeros(128, 32, **BF), w, w_grad=False)


@pytest.mark.gpu
def test_gradients_without_the_rows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    idx = torch.topk(rand(90, 7).float(), 2, dim=1).indices.int().contiguous()
    p = cs.Plan(90, 8, 7, 2, 1).route(idx)
    gy, x, w, pre = rand(180, 40), rand(180, 72), rand(7, 80, 72), rand(180, 80)
    want = p.expert_linear_backward(gy, x, w, pre, "swiglu", bias_grad=True)
    gx, gw, gb = p.expert_linear_backward(gy, None, w, pre, "swiglu", bias_grad=True, w_grad=False)
    assert gw is None and torch.equal(gx, want[0]) and torch.equal(gb, want[2])
    _, _, gb = p.expert_linear_backward(gy, None, w, pre, "swiglu", True, x_grad=False, w_grad=False)
    assert torch.equal(gb, want[2])
