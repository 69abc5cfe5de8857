"""The C ABI of include/moe_block.h and its Python binding on the host (CPU, no GPU needed):
exports, and every refusal that comes before a launch."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import block_ref
import combine_shuffling_amd as cs
from combine_shuffling_amd import _abi

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_block.h")
BAD, UNSUPPORTED = _abi.ERR_INVALID_ARGUMENT, _abi.ERR_UNSUPPORTED
vp = ctypes.c_void_p


def plan(T=64, H=64, E=8, k=2, R=2, **kw):
    return cs.Plan(T, H, E, k, R, **kw)


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(_abi.BLOCK_EXPORTS)
    for n in names:
        assert hasattr(_abi.lib(), n), n


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "moe_block.h"\nint main(void) { return MOE_BLOCK_KERNEL_END != %d; }\n'
                   % _abi.BLOCK_KERNELS.stop)
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.dirname(HEADER), str(src),
                    "-o", exe], check=True, timeout=120)
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_kernel_names_are_the_kernels_symbols():
    csrc = os.path.join(os.path.dirname(HEADER), "..", "combine_shuffling_amd", "csrc")
    text = "".join(open(os.path.join(csrc, f)).read() for f in os.listdir(csrc)
                   if f.endswith((".hip", ".h")))
    kernels = set(re.findall(r"void\s+(\w+_kernel)\s*\(", text))
    names = [_abi.kernel_name(i) for i in _abi.BLOCK_KERNELS]
    assert len(set(names)) == len(names) and set(names) <= kernels
    assert _abi.BLOCK_KERNELS.start > _abi.KERNEL_COUNT
    for i in (_abi.BLOCK_KERNELS.start - 1, _abi.BLOCK_KERNELS.stop):
        assert _abi.kernel_name(i) == "?"


# ---- the norm

def norm(p, cfg=(0, 1e-5, 0, 0), x=16, residual=None, gamma=16, beta=16, y=16, total=None, stats=None):
    c = _abi.NormConfig(*cfg)
    return _abi.lib().moe_norm(p._h, ctypes.byref(c), vp(x), vp(residual), vp(gamma), vp(beta), vp(y),
                               vp(total), vp(stats), None)


def norm_backward(p, cfg=(0, 1e-5, 0, 0), gy=16, total=16, stats=16, gamma=16, gt=None, gx=16, gg=16,
                  gb=16, ws=256):
    c = _abi.NormConfig(*cfg)
    return _abi.lib().moe_norm_backward(p._h, ctypes.byref(c), vp(gy), vp(total), vp(stats), vp(gamma),
                                        vp(gt), vp(gx), vp(gg), vp(gb), vp(ws), None)


CONFIGS = [((2, 1e-5, 0, 0), BAD), ((-1, 1e-5, 0, 0), BAD), ((0, -1e-9, 0, 0), BAD),
           ((0, float("nan"), 0, 0), BAD), ((0, float("inf"), 0, 0), BAD), ((0, 0.0, 2, 0), BAD),
           ((0, 0.0, 0, 2), BAD), ((0, 0.0, -1, 0), BAD)]


@pytest.mark.parametrize("cfg,want", CONFIGS)
def test_norm_config_refusals(cfg, want):
    p = plan()
    assert norm(p, cfg) == norm_backward(p, cfg) == want
    assert _abi.lib().moe_norm_backward_workspace_bytes(p._h, ctypes.byref(_abi.NormConfig(*cfg))) == 0


def test_norm_width_limit():
    good = _abi.NormConfig(0, 0.0, 0, 0)
    for H, ok in ((16384, True), (16392, False)):
        p = plan(T=0, H=H)
        assert norm(p) == (_abi.OK if ok else UNSUPPORTED)
        if not ok:
            assert norm_backward(p) == UNSUPPORTED
            assert _abi.lib().moe_norm_backward_workspace_bytes(p._h, ctypes.byref(good)) == 0


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=8), dict(y=None), dict(y=24), dict(gamma=4), dict(beta=8),
    dict(residual=8), dict(residual=16, total=8), dict(total=16),       # a total without a residual
    dict(stats=4),
])
def test_norm_pointer_refusals(kw):
    assert norm(plan(), **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(gy=None), dict(gy=8), dict(total=None), dict(total=8), dict(stats=None), dict(stats=4),
    dict(gamma=8), dict(gt=8), dict(gx=8), dict(gg=8), dict(gb=8), dict(ws=128), dict(ws=None),
])
def test_norm_backward_pointer_refusals(kw):
    assert norm_backward(plan(T=5000, H=2048), **kw) == BAD


def test_norm_without_plan_or_config():
    L, c = _abi.lib(), _abi.NormConfig(0, 0.0, 0, 0)
    assert norm_backward(plan(), gx=None, gg=None, gb=None) == _abi.OK      # nothing is wanted
    assert L.moe_norm(None, ctypes.byref(c), vp(16), None, None, None, vp(16), None, None, None) == BAD
    assert L.moe_norm(plan()._h, None, vp(16), None, None, None, vp(16), None, None, None) == BAD
    assert L.moe_norm_backward(None, ctypes.byref(c), vp(16), vp(16), vp(16), None, None, vp(16), None,
                               None, None, None) == BAD


def test_norm_workspace_bytes():
    # two sets of float32 partial sums of up to 256 blocks; none where one block is enough
    size = lambda T, H: _abi.lib().moe_norm_backward_workspace_bytes(  # noqa: E731
        plan(T=T, H=H)._h, ctypes.byref(_abi.NormConfig(0, 0.0, 0, 0)))
    assert size(0, 64) == size(1, 2048) == size(4, 8192) == 0
    assert size(100000, 2048) == 2 * 256 * 2048 * 4
    assert size(5, 8192) == 2 * 5 * 8192 * 4
    assert size(100000, 72) % 256 == 0


def test_norm_binding_refusals():
    p = plan()
    x, v = torch.zeros(64, 64), torch.zeros(64)
    st = torch.zeros(64, 2)
    bf = x.bfloat16()
    for call, match in [
        (lambda: p.norm(x, kind="batch"), "kind"),
        (lambda: p.norm(x[:, :32]), "shape"),
        (lambda: p.norm(x.double()), "dtype"),
        (lambda: p.norm(x.t()), "contiguous"),
        (lambda: p.norm(x, v.bfloat16()), "gamma"),
        (lambda: p.norm(x, v, v[:32]), "beta"),
        (lambda: p.norm(x, v, v, bf), "residual"),
        (lambda: p.norm(x, v, total=x), "total"),
        (lambda: p.norm(x, v, out_dtype=torch.float16), "out_dtype"),
        (lambda: p.norm(x, v, y=x, out_dtype=torch.float32), "shares"),
        (lambda: p.norm(x, v, y=bf, out_dtype=torch.float32), "y has"),
        (lambda: p.norm(x, v, residual=x.clone(), total=x), "shares"),
        (lambda: p.norm(x, v, stats=st[:, 0]), "stats"),
        (lambda: p.norm(x, v), "GPU"),
        (lambda: p.norm_backward(bf, x, st[:, :1]), "stats"),
        (lambda: p.norm_backward(bf[:2], x, st), "grad_y"),
        (lambda: p.norm_backward(bf, x, st, x), "gamma"),
        (lambda: p.norm_backward(bf, x, st, v, grad_total=bf), "grad_total"),
        (lambda: p.norm_backward(bf, x, st, v, grad_x=x), "shares"),
        (lambda: p.norm_backward(bf, x, st, v, grad_gamma=v), "shares"),
        (lambda: p.norm_backward(bf, x, st, v, grad_x=bf.clone()), "grad_x"),
        (lambda: p.norm_backward(bf, x, st, v, grad_beta=v.double()), "grad_beta"),
        (lambda: p.norm_backward(bf, x, st, v, kind="group"), "kind"),
        (lambda: p.norm_backward(bf, x, st, v), "GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    big = plan(T=5000, H=64)
    x = torch.zeros(5000, 64)
    with pytest.raises(ValueError, match="workspace too small"):
        big.norm_backward(x, x.clone(), torch.zeros(5000, 2), workspace=torch.zeros(64))


def test_norm_gradient_definition_against_differences():
    # The definition's own gradient, by central differences of the definition, in 64 bits.
    rng = np.random.default_rng(3)
    T, H, eps = 3, 24, 1e-3
    x, gamma, beta = rng.normal(size=(T, H)) + 0.5, rng.normal(size=H), rng.normal(size=H)
    gy, gt = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    for rms in (False, True):
        f = lambda x, g, b: (block_ref.norm(x, g, b, rms, eps)["y"][0] * gy).sum() + (x * gt).sum()  # noqa: E731
        r = block_ref.norm(x, gamma, beta, rms, eps)
        stats = np.stack([r["mean"][0], r["rstd"][0]], 1)
        got = block_ref.norm_backward(gy, x, stats, gamma, gt, rms)
        args = [x, gamma, beta]
        for i, name in enumerate(("grad_x", "grad_gamma", "grad_beta")):
            want = np.zeros_like(args[i])
            for at in np.ndindex(want.shape):
                d = np.zeros_like(args[i])
                d[at] = 1e-5
                up, down = list(args), list(args)
                up[i], down[i] = args[i] + d, args[i] - d
                want[at] = (f(*up) - f(*down)) / 2e-5
            # differences: third derivatives times 1e-10, and 2^-52 of sums of 72 terms over 1e-5
            assert np.abs(got[name][0] - want).max() < 1e-6, (rms, name)


# ---- 4-bit weights

def w4cfg(E=8, Z=64, K=64, fmt=0, group=128):
    return _abi.Weights4Config(E, Z, K, fmt, group)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), BAD), (dict(E=-1), BAD), (dict(Z=0), BAD), (dict(Z=12), BAD), (dict(K=0), BAD),
    (dict(K=-8), BAD), (dict(K=60), BAD), (dict(fmt=2), BAD), (dict(fmt=-1), BAD), (dict(group=0), BAD),
    (dict(group=16), BAD), (dict(group=96), BAD), (dict(group=256), BAD), (dict(group=-32), BAD),
    (dict(fmt=1, group=64), BAD), (dict(fmt=1, group=128), BAD),
    (dict(E=1025), UNSUPPORTED), (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(Z=(1 << 20) + 8), UNSUPPORTED),
    (dict(Z=1 << 15, K=1 << 15), UNSUPPORTED),
])
def test_weights4_config_refusals(kw, want):
    L, c = _abi.lib(), ctypes.byref(w4cfg(**kw))
    assert L.moe_weights4_bytes(c) == 0
    assert L.moe_weights4_pack(c, vp(256), vp(256), vp(256), None) == want
    assert L.moe_weights4_quantize(c, vp(256), vp(256), None) == want
    assert L.moe_weights4_unpack(c, vp(256), vp(256), 0, None) == want
    e = _abi.ExpertConfig(64, 64, 0)
    assert L.moe_expert_linear4(plan()._h, ctypes.byref(e), c, vp(256), vp(256), None, None, vp(256),
                                None) == want


def test_weights4_pointer_refusals():
    L, c = _abi.lib(), ctypes.byref(w4cfg())
    m = ctypes.byref(w4cfg(fmt=1, group=32))
    assert L.moe_weights4_pack(None, vp(256), vp(256), vp(256), None) == BAD
    for codes, scales, packed in ((None, 256, 256), (8, 256, 256), (256, None, 256), (256, 257, 256),
                                  (256, 256, None), (256, 256, 128)):
        assert L.moe_weights4_pack(c, vp(codes), vp(scales), vp(packed), None) == BAD
    assert L.moe_weights4_pack(m, vp(256), None, vp(256), None) == BAD
    for w, packed in ((None, 256), (8, 256), (256, None), (256, 16)):
        assert L.moe_weights4_quantize(c, vp(w), vp(packed), None) == BAD
        assert L.moe_weights4_unpack(c, vp(packed), vp(w), 0, None) == BAD
    assert L.moe_weights4_unpack(c, vp(256), vp(256), 2, None) == BAD
    assert L.moe_weights4_bytes(None) == 0


def test_weights4_bytes():
    size = lambda **kw: _abi.lib().moe_weights4_bytes(ctypes.byref(w4cfg(**kw)))  # noqa: E731
    # blocks of 128 weights of a row in 64 bytes, and their scales
    assert size(E=2, Z=64, K=256) == 2 * 64 * 128 + 2 * 64 * 2 * 2
    assert size(E=2, Z=64, K=256, group=32) == 2 * 64 * 128 + 2 * 64 * 8 * 2
    assert size(E=2, Z=64, K=256, fmt=1, group=32) == 2 * 64 * 128 + 2 * 64 * 8
    assert size(E=2, Z=64, K=136) == size(E=2, Z=64, K=256)
    assert size(E=1, Z=8, K=8) == 1024 + 256     # 16 rows


def test_expert_linear4_refusals():
    L, p = _abi.lib(), plan()

    def call(cfg=(64, 64, 0), w4=None, x=16, packed=256, bias=None, residual=None, y=16, plan_=p._h):
        c = ctypes.byref(_abi.ExpertConfig(*cfg)) if cfg else None
        return L.moe_expert_linear4(plan_, c, ctypes.byref(w4 or w4cfg()), vp(x), vp(packed), vp(bias),
                                    vp(residual), vp(y), None)

    assert call() == _abi.ERR_PLAN_NOT_ROUTED
    assert call(plan_=None) == call(cfg=None) == BAD
    assert L.moe_expert_linear4(p._h, ctypes.byref(_abi.ExpertConfig(64, 64, 0)), None, vp(16), vp(256),
                                None, None, vp(16), None) == BAD
    for cfg, w4 in [((64, 64, 6), None), ((64, 64, -1), None), ((64, 0, 0), None), ((64, 12, 0), None),
                    ((72, 64, 0), None), ((64, 72, 0), None), ((64, 64, 4), None),      # Z = 2N when gated
                    ((64, 64, 0), w4cfg(E=7)), ((64, 64, 0), w4cfg(Z=128))]:
        assert call(cfg, w4) == BAD, cfg
    assert call((64, 32, 4)) == _abi.ERR_PLAN_NOT_ROUTED


def test_weights4_binding_refusals():
    codes = torch.zeros(8, 64, 32, dtype=torch.uint8)
    bf = torch.zeros(8, 64, 1, dtype=torch.bfloat16)
    for call, match in [
        (lambda: cs.pack_experts4(codes, bf, "int8"), "format"),
        (lambda: cs.pack_experts4(codes[0], bf), "expected"),
        (lambda: cs.pack_experts4(codes.int(), bf), "codes"),
        (lambda: cs.pack_experts4(codes[:, :, ::2], bf), "contiguous"),
        (lambda: cs.pack_experts4(codes, bf, group=0), "not supported"),
        (lambda: cs.pack_experts4(codes, bf, group=48), "not supported"),
        (lambda: cs.pack_experts4(codes[:, :, :3].contiguous(), bf), "not supported"),
        (lambda: cs.pack_experts4(codes, bf, group=32), "scales"),
        (lambda: cs.pack_experts4(codes, bf.float()), "scales"),
        (lambda: cs.pack_experts4(codes, torch.zeros(8, 64, 2, dtype=torch.bfloat16), "e2m1", 32), "scales"),
        (lambda: cs.pack_experts4(codes, bf, "e2m1", 128), "not supported"),
        (lambda: cs.pack_experts4(codes, bf), "GPU"),
        (lambda: cs.quantize_experts4(torch.zeros(8, 64, 64)), "dtype"),
        (lambda: cs.quantize_experts4(torch.zeros(8, 64)), "expected"),
        (lambda: cs.quantize_experts4(torch.zeros(8, 64, 64, dtype=torch.bfloat16).transpose(1, 2)),
         "contiguous"),
        (lambda: cs.quantize_experts4(torch.zeros(8, 64, 64, dtype=torch.bfloat16)), "GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    p = plan()
    w4 = cs.ExpertWeights4(8, 32, 64, "int4", 128, torch.device("cpu"))
    with pytest.raises(ValueError, match="GPU"):
        w4.values()
    with pytest.raises(ValueError, match="dtype"):
        w4.values(torch.float16)
    x = torch.zeros(128, 64, dtype=torch.bfloat16)
    with pytest.raises(cs.MoeError):       # not routed
        p.expert_linear4(x, w4)
    p.device = torch.device("cpu")         # as if routed: the checks come before any launch
    out = torch.zeros(128, 32, dtype=torch.bfloat16)
    for call, match in [
        (lambda: p.expert_linear4(x, w4, activation="tanh"), "activation"),
        (lambda: p.expert_linear4(x, cs.ExpertWeights4(7, 32, 64, "int4", 128, p.device)), "experts"),
        (lambda: p.expert_linear4(x, cs.ExpertWeights4(8, 40, 64, "int4", 128, p.device),
                                  activation="swiglu"), "halves"),
        (lambda: p.expert_linear4(x[:, :32], w4), "x has"),
        (lambda: p.expert_linear4(x.float(), w4), "x has"),
        (lambda: p.expert_linear4(x, w4, bias=torch.zeros(8, 64)), "bias"),
        (lambda: p.expert_linear4(x, w4, residual=x), "residual"),
        (lambda: p.expert_linear4(x, w4, y=x.clone()), "y has"),
        (lambda: p.expert_linear4(x, w4, residual=out, y=out), "shares"),
        (lambda: p.expert_linear4(x, w4), "GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError):
        p.expert_linear4(x, torch.zeros(8, 32, 64, dtype=torch.bfloat16))


def test_quantizer_definition():
    # Hand-made groups: codes and scales as the formats' rules give them.
    w = np.zeros((1, 3, 32))
    w[0, 0, :4] = [7, -7, 3.5, 0.5]            # scale 1: halves go to the even code
    w[0, 1, :4] = [-14, 3, 5, 6.9]             # scale 2: 1.5 and 2.5 both go to 2
    codes, scales = block_ref.quantize4(w, "int4", 32)
    assert scales[0].tolist() == [[1.0], [2.0], [0.0]]
    assert codes[0, :, :4].tolist() == [[15, 1, 12, 8], [1, 10, 10, 11], [8] * 4]
    w[0, 0, :8] = [6, -6, 5, 3.5, 2.5, 0.25, 0.75, -1.25]
    w[0, 1, :2] = [6.25, 0.1]
    codes, scales = block_ref.quantize4(w, "e2m1", 32)
    assert scales[0].tolist() == [[127], [128], [127]]
    assert codes[0, 0, :8].tolist() == [7, 15, 6, 6, 4, 0, 2, 10]
