"""The buffer of packed 4-bit weights is a public attribute, in whose place a program may put one that it
saved: the calls that read it take one of the weights' own size and kind only (CPU, no GPU needed)."""

import pytest
import torch

import combine_shuffling_amd as cs

CPU = torch.device("cpu")


def weights(E=8, Z=32, K=64):
    return cs.ExpertWeights4(E, Z, K, "int4", 128, CPU)


def others(w4):
    size = w4.packed.numel()
    return {
        "shorter": torch.zeros(size - 256, dtype=torch.uint8),
        "longer": torch.zeros(size + 256, dtype=torch.uint8),
        "of another layout": cs.ExpertWeights4(8, 32, 64, "e2m1", 32, CPU).packed,
        "of another shape": torch.zeros(2, size // 2, dtype=torch.uint8),
        "of another type": torch.zeros(size, dtype=torch.int8),
        "elsewhere": torch.zeros(size, dtype=torch.uint8, device="meta"),
        "with gaps": torch.zeros(2 * size, dtype=torch.uint8)[::2],
    }


@pytest.mark.parametrize("kind", list(others(weights())))
def test_another_buffer_is_refused(kind):
    w4 = weights()
    x = torch.zeros(128, 64, dtype=torch.bfloat16)
    plan = cs.Plan(64, 64, 8, 2, 2)
    plan.device = CPU                       # as if routed: the checks come before any launch
    w4.packed = others(w4)[kind]
    with pytest.raises(ValueError, match="packed"):
        plan.expert_linear4(x, w4)
    with pytest.raises(ValueError, match="packed"):
        w4.values()


def test_a_saved_buffer_is_taken():
    # (Past the checks: the GPU is asked for.)
    w4 = weights()
    w4.packed = w4.packed.clone()
    plan = cs.Plan(64, 64, 8, 2, 2)
    plan.device = CPU
    with pytest.raises(ValueError, match="GPU"):
        plan.expert_linear4(torch.zeros(128, 64, dtype=torch.bfloat16), w4)
    with pytest.raises(ValueError, match="GPU"):
        w4.values()


def test_not_a_tensor():
    w4 = weights()
    w4.packed = None
    with pytest.raises(TypeError, match="packed"):
        w4.values()


@pytest.mark.parametrize("name", ["experts", "rows", "in_features"])
def test_sizes_are_the_buffers_own(name):
    w4 = weights()
    assert (w4.experts, w4.rows, w4.in_features) == (8, 32, 64)
    with pytest.raises(AttributeError):
        setattr(w4, name, 16)
