"""The layer's C ABI (include/moe_layer.h) and its Python binding on the host (CPU, no GPU
needed): exports, and every refusal that comes before a launch."""

import ctypes
import os
import re

import pytest
import torch

import combine_shuffling_amd as cs
from combine_shuffling_amd import _abi

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_layer.h")
BAD, UNROUTED, UNSUPPORTED = (_abi.ERR_INVALID_ARGUMENT, _abi.ERR_PLAN_NOT_ROUTED,
                              _abi.ERR_UNSUPPORTED)
vp = ctypes.c_void_p


def plan(T=64, H=64, E=8, k=2, R=2, **kw):
    return cs.Plan(T, H, E, k, R, **kw)


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(_abi.LAYER_EXPORTS)
    for n in names:
        assert hasattr(_abi.lib(), n), n


def test_header_compiles_as_c(tmp_path):
    import subprocess

    src = tmp_path / "t.c"
    src.write_text('#include "moe_layer.h"\nint main(void) { return MOE_LAYER_KERNEL_END != %d; }\n'
                   % _abi.KERNEL_COUNT)
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.dirname(HEADER), str(src),
                    "-o", exe], check=True, timeout=120)
    assert subprocess.run([exe], timeout=60).returncode == 0


def router(p, cfg=(0, 1, 0, 1.0), logits=16, dtype=1, bias=None, idx=16, w=16):
    c = _abi.RouterConfig(*cfg)
    return _abi.lib().moe_router(p._h, ctypes.byref(c), vp(logits), dtype, vp(bias), vp(idx), vp(w),
                                 None)


@pytest.mark.parametrize("kw", [
    dict(cfg=(2, 1, 0, 1.0)), dict(cfg=(-1, 1, 0, 1.0)),              # unknown score
    dict(cfg=(0, 1, -1, 1.0)), dict(cfg=(0, 1, 3, 1.0)),              # nodes outside 0..N
    dict(cfg=(0, 1, 0, float("nan"))), dict(cfg=(0, 1, 0, float("inf"))),
    dict(dtype=2), dict(dtype=-1),
    dict(logits=None), dict(idx=None), dict(w=None),
    dict(logits=18), dict(idx=18), dict(w=17), dict(bias=18), dict(dtype=0, logits=17),
])
def test_router_refusals(kw):
    p = plan(R=2, ranks_per_node=1)
    assert router(p, **kw) == BAD
    c = _abi.RouterConfig(*kw.get("cfg", (0, 1, 0, 1.0)))
    if "bias" not in kw:
        st = _abi.lib().moe_router_backward(p._h, ctypes.byref(c), vp(kw.get("logits", 16)),
                                            kw.get("dtype", 1), vp(kw.get("idx", 16)),
                                            vp(kw.get("w", 16)), vp(16), None)
        assert st == BAD


def test_router_node_limits():
    # 10 experts on 4 one-rank nodes (3, 3, 2, 2): the smallest node holds 2
    p = plan(E=10, k=3, R=4, ranks_per_node=1)
    assert router(p, cfg=(0, 1, 1, 1.0)) == BAD
    # 65 nodes are past the limit, but only where nodes are chosen
    p = plan(T=0, E=65, k=2, R=65, ranks_per_node=1)
    assert router(p, cfg=(0, 1, 1, 1.0)) == UNSUPPORTED
    assert router(p, cfg=(0, 1, 0, 1.0)) == _abi.OK          # T = 0: nothing is launched
    assert _abi.lib().moe_router(None, None, None, 0, None, None, None, None) == BAD


def test_router_backward_pointers():
    p, c = plan(), _abi.RouterConfig(0, 1, 0, 1.0)
    f = _abi.lib().moe_router_backward
    assert f(p._h, ctypes.byref(c), vp(16), 1, vp(16), vp(16), None, None) == BAD
    assert f(p._h, ctypes.byref(c), vp(16), 1, vp(16), vp(16), vp(18), None) == BAD
    assert f(p._h, None, vp(16), 1, vp(16), vp(16), vp(16), None) == BAD


def test_calls_before_route_are_refused():
    L, p = _abi.lib(), plan()
    c = _abi.ExpertConfig(64, 64, 0)
    assert L.moe_dispatch_backward(p._h, vp(16), vp(16), 0, None) == UNROUTED
    assert L.moe_combine_backward(p._h, vp(16), 0, vp(16), vp(16), vp(16), vp(16), None) == UNROUTED
    assert L.moe_expert_linear(p._h, ctypes.byref(c), vp(16), vp(16), None, None, vp(16), None,
                               None) == UNROUTED
    assert L.moe_expert_linear_backward(p._h, ctypes.byref(c), vp(16), vp(16), vp(16), None, vp(16),
                                        vp(16), 0, None, vp(256), None) == UNROUTED
    for f in (L.moe_dispatch_backward,):
        assert f(None, vp(16), vp(16), 0, None) == BAD
    assert L.moe_combine_backward(None, vp(16), 0, vp(16), vp(16), vp(16), vp(16), None) == BAD


@pytest.mark.parametrize("cfg,want", [
    ((0, 64, 0), BAD), ((64, 0, 0), BAD), ((-8, 64, 0), BAD),
    ((12, 64, 0), BAD), ((64, 12, 0), BAD),            # not multiples of 8
    ((64, 64, 6), BAD), ((64, 64, -1), BAD),           # unknown activation
    (((1 << 20) + 8, 64, 0), UNSUPPORTED), ((64, (1 << 20) + 8, 0), UNSUPPORTED),
    ((64, (1 << 19) + 8, 4), UNSUPPORTED),             # gated: 2N rows
    ((1 << 15, 1 << 15, 0), UNSUPPORTED),              # one expert's weight reaches 2^30 elements
])
def test_expert_config_refusals(cfg, want):
    L, p = _abi.lib(), plan()
    c = _abi.ExpertConfig(*cfg)
    assert L.moe_expert_linear(p._h, ctypes.byref(c), vp(16), vp(16), None, None, vp(16), None,
                               None) == want
    assert L.moe_expert_linear_backward(p._h, ctypes.byref(c), vp(16), vp(16), vp(16), vp(16), vp(16),
                                        vp(16), 0, None, vp(256), None) == want
    assert L.moe_expert_backward_workspace_bytes(p._h, ctypes.byref(c)) == 0


def test_backward_workspace_bytes():
    # grad_z (with an activation) and 32-row partial sums of every column
    p = plan(T=100, E=8, k=2)
    L = _abi.lib()
    size = lambda *c: L.moe_expert_backward_workspace_bytes(p._h, ctypes.byref(_abi.ExpertConfig(*c)))  # noqa: E731
    slots = 200 // 32 + 8
    assert size(64, 64, 0) == slots * 64 * 4
    assert size(64, 64, 4) == 200 * 128 * 2 + slots * 128 * 4
    assert size(64, 40, 2) % 256 == 0
    # banded: every band has slots of its own for its experts
    p = plan(T=1024, band_tokens=256)
    assert size(64, 64, 0) == (2048 // 32 + 4 * 8) * 64 * 4
    assert L.moe_expert_linear(p._h, None, vp(16), vp(16), None, None, vp(16), None, None) == BAD


def test_kernel_names():
    names = [_abi.kernel_name(i) for i in range(22, _abi.KERNEL_COUNT)]
    assert names == ["router_kernel", "router_grad_kernel", "dispatch_grad_kernel",
                     "combine_grad_kernel", "expert_rows_kernel", "expert_few_rows_kernel",
                     "expert_rows_grad_kernel",
                     "expert_wgrad_kernel", "expert_grads_kernel",
                     "expert_act_grad_kernel", "expert_bias_sum_kernel"]


# ---- the Python binding's own checks

def test_binding_refuses_before_route():
    p = plan()
    x = torch.zeros(128, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, 64, dtype=torch.bfloat16)
    for call in (lambda: p.dispatch_backward(x), lambda: p.combine_backward(x, x, x),
                 lambda: p.expert_linear(x, w), lambda: p.expert_linear_backward(x, x, w)):
        with pytest.raises(cs.MoeError) as e:
            call()
        assert e.value.status == UNROUTED


def test_binding_refuses_cpu_tensors_and_wrong_arguments():
    p = plan()
    logits = torch.zeros(64, 8)
    with pytest.raises(ValueError, match="GPU"):
        p.router(logits)
    with pytest.raises(ValueError, match="score"):
        p.router(logits, score="relu")
    with pytest.raises(ValueError, match="shape"):
        p.router(torch.zeros(64, 9))
    with pytest.raises(ValueError, match="dtype"):
        p.router(logits.double())
    with pytest.raises(ValueError, match="contiguous"):
        p.router(torch.zeros(8, 64).t())
    with pytest.raises(ValueError, match="bias"):
        p.router(logits, bias=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="grad_w"):
        p.router_backward(logits, torch.zeros(64, 2, dtype=torch.int32), torch.zeros(64, 3))


def test_binding_checks_expert_arguments():
    p = plan()
    p.device = torch.device("cpu")   # as if routed: the checks come before any launch
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros(128, 64, **bf), torch.zeros(8, 32, 64, **bf)
    gy = torch.zeros(128, 32, **bf)
    for call, match in [
        (lambda: p.expert_linear(x, w, activation="tanh"), "activation"),
        (lambda: p.expert_linear(x, w[0]), "expected"),
        (lambda: p.expert_linear(x, torch.zeros(7, 32, 64, **bf)), "shape"),
        (lambda: p.expert_linear(x, w.float()), "dtype"),
        (lambda: p.expert_linear(x[:, :32], w), "shape"),
        (lambda: p.expert_linear(x, w.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
        (lambda: p.expert_linear(x, w, bias=torch.zeros(8, 32, **bf)), "bias"),
        (lambda: p.expert_linear(x, w, residual=torch.zeros(128, 64, **bf)), "residual"),
        (lambda: p.expert_linear(x, torch.zeros(8, 33, 64, **bf), activation="swiglu"), "even"),
        (lambda: p.expert_linear_backward(gy, x, w, activation="silu"), "pre"),
        (lambda: p.expert_linear_backward(gy, x, w, pre=gy.float(), activation="silu"), "pre"),
        (lambda: p.expert_linear_backward(gy, x, w, grad_w_dtype=torch.float16), "grad_w_dtype"),
        (lambda: p.expert_linear_backward(gy, x, w, workspace=torch.zeros(1)), "workspace"),
        (lambda: p.expert_linear(x, w), "GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError):
        p.expert_linear(x, None)


def test_binding_refuses_outputs_that_share_memory():
    p = plan()
    p.device = torch.device("cpu")   # as if routed
    bf = dict(dtype=torch.bfloat16)
    logits, x, w = torch.zeros(64, 8), torch.zeros(128, 64, **bf), torch.zeros(8, 64, 64, **bf)
    pre, go, k32 = torch.zeros(128, 64, **bf), torch.zeros(64, 64, **bf), torch.zeros(64, 2)
    both = torch.zeros(128, 64, **bf)
    for call in (lambda: p.router(logits, topk_w=logits.view(-1)[:128].view(64, 2)),
                 lambda: p.router(logits, topk_idx=k32.view(torch.int32), topk_w=k32),
                 lambda: p.router_backward(logits, k32.int(), k32, grad_logits=logits),
                 lambda: p.dispatch_backward(x, grad_x=x[:64]),
                 lambda: p.combine_backward(go, x, k32, grad_y=x),
                 lambda: p.combine_backward(go, x, k32, grad_w=k32),
                 lambda: p.expert_linear(x, w, residual=pre, y=pre),
                 lambda: p.expert_linear(x, w, y=both, pre=both),
                 lambda: p.expert_linear(x, w, y=x),
                 lambda: p.expert_linear_backward(pre, x, w, grad_x=x),
                 lambda: p.expert_linear_backward(pre, x, w, grad_w=w),
                 lambda: p.expert_linear_backward(both, x, w, workspace=both.view(torch.uint8))):
        with pytest.raises(ValueError, match="shares memory"):
            call()
    # neighbours in one buffer are apart
    with pytest.raises(ValueError, match="GPU"):
        p.dispatch_backward(x, grad_x=torch.zeros(192, 64, **bf)[128:])
    buffer = torch.zeros(192, 64, **bf)
    with pytest.raises(ValueError, match="GPU"):
        p.dispatch_backward(buffer[:128], grad_x=buffer[128:])


def test_binding_checks_the_workspace():
    p = plan()
    p.device = torch.device("cpu")
    bf = dict(dtype=torch.bfloat16)
    x, w, gy = torch.zeros(128, 64, **bf), torch.zeros(8, 32, 64, **bf), torch.zeros(128, 32, **bf)
    with pytest.raises(ValueError, match="contiguous"):   # many elements, one byte of memory
        p.expert_linear_backward(gy, x, w, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(ValueError, match="is on"):
        p.expert_linear_backward(gy, x, w, workspace=torch.empty(1 << 20, device="meta"))
    with pytest.raises(TypeError):
        p.expert_linear_backward(gy, x, w, workspace=4096)


def test_binding_refuses_a_stream_of_another_device():
    class Elsewhere:
        device = torch.device("cuda", 1)
    p = plan()
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        p.router(torch.zeros(64, 8), stream=Elsewhere())
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        cs.router_backward(p, torch.zeros(64, 8), torch.zeros(64, 2, dtype=torch.int32),
                           torch.zeros(64, 2), stream=Elsewhere())
