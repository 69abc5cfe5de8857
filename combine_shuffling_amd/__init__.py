"""MI355X (gfx950) MoE expert-parallel shuffle.

A thin binding over the C ABI of ``libmoeshuffle.so`` (include/moe_shuffle.h,
include/moe_layer.h and include/moe_block.h): the same calls, with torch tensors
for device memory and torch's current stream.  Every step of the shuffle runs in
the library's HIP kernels; this module only checks shapes and passes pointers.

    plan = route_plan(topk_idx, num_experts=E, num_ranks=R, hidden=H,
                      ranks_per_node=G, node_dedup=False)
    recv, staging = dispatch(plan, x)           # x: [T, H] bf16 on the GPU
    out = combine(plan, y, topk_w)              # y: [T*k, H] bf16, receive layout

Banded plans (band_tokens > 0) route each band of consecutive tokens as its
own batch; ``Plan.pipeline`` runs route, dispatch and combine of every band
in one persistent launch.

Around the shuffle stand the other operators of a Mixture-of-Experts layer and
the layer's gradients:

    plan = Plan(T, H, E, k, R)
    idx, w = router(plan, logits)               # gate logits [T, E] -> ids, combine weights
    plan.route(idx)
    recv, _ = dispatch(plan, x)
    h, pre = expert_linear(plan, recv, w1, activation="swiglu", save_pre=True)
    y, _ = expert_linear(plan, h, w2)
    out = combine(plan, y, w)

    grad_y, grad_w = combine_backward(plan, grad_out, y, w)
    grad_h, grad_w2, _ = expert_linear_backward(plan, grad_y, h, w2)
    grad_recv, grad_w1, _ = expert_linear_backward(plan, grad_h, recv, w1, pre, "swiglu")
    grad_x = dispatch_backward(plan, grad_recv)
    grad_logits = router_backward(plan, logits, idx, grad_w)

Before it stands the norm of the residual stream, and a model that only answers
may keep its experts' weights in 4 bits:

    h, stream, stats = norm(plan, x, gamma, residual=delta, save_stats=True)
    grad_x, grad_gamma, _ = norm_backward(plan, grad_h, stream, stats, gamma)

    w4 = quantize_experts4(w1, "int4", 128)     # once; pack_experts4 for a checkpoint's codes
    h = expert_linear4(plan, recv, w4, activation="swiglu")

Outputs may be given to these calls; they share no memory with other arguments.
"""

from __future__ import annotations

import ctypes
import functools

import numpy as np
import torch

from . import _abi
from ._abi import MoeError, ITEM  # noqa: F401

__all__ = ["Plan", "MoeError", "expert_partition", "route_plan", "dispatch", "combine",
           "dispatch_fp8", "combine_fp8", "combine_hier", "pipeline", "router", "router_backward",
           "expert_linear", "expert_linear_backward", "combine_backward", "dispatch_backward", "norm",
           "norm_backward", "ExpertWeights4", "pack_experts4", "quantize_experts4", "expert_linear4"]


def expert_partition(num_experts: int, num_ranks: int) -> list[int]:
    """moe_expert_partition: rank d holds experts [lo[d], lo[d+1])."""
    lo = (ctypes.c_int32 * (num_ranks + 1))() if num_ranks > 0 else (ctypes.c_int32 * 1)()
    _abi.check(_abi.lib().moe_expert_partition(num_experts, num_ranks, lo), "moe_expert_partition")
    return list(lo)


def _stream_handle(device: torch.device, stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, shape, dtypes, name: str, device) -> None:
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and
            t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_OUT_CODE = {torch.bfloat16: _abi.OUT_BF16, torch.float32: _abi.OUT_F32}


def _out_code(dtype, name: str) -> int:
    if dtype not in _OUT_CODE:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32")
    return _OUT_CODE[dtype]


def _out(t: torch.Tensor | None, shape, dtype, name: str, device) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:   # torch.empty takes 0.4 us more, a twentieth of a small call
        stride = (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1)
        return torch.empty_strided(shape, stride, dtype=dtype, device=device)
    _need(t, shape, (dtype,), name, device)
    return t


def _vector(t: torch.Tensor | None, n: int, name: str, device) -> torch.Tensor:
    """The caller's float32 output [n], checked, or a new one."""
    if t is None:
        return torch.empty_strided((n,), (1,), dtype=torch.float32, device=device)
    _need(t, (n,), _F32, name, device)
    return t


def _apart(given, others) -> None:
    """The outputs that the caller gives share no memory with each other or with an input."""
    for i, t in enumerate(given):
        if t is None:
            continue
        end = t.data_ptr() + t.numel() * t.element_size()
        for o in (*given[i + 1:], *others):
            if (o is not None and o.data_ptr() < end and
                    t.data_ptr() < o.data_ptr() + o.numel() * o.element_size()):
                raise ValueError("an output shares memory with another argument")


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _on_stream(method):
    """A call that also takes stream=: it then runs with that stream current, so that what it
    allocates belongs to that stream too.  The stream has to be one of the tensors' device."""
    @functools.wraps(method)
    def call(*args, stream=None, **kw):
        if stream is None:
            return method(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.device != stream.device:
                raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
        with torch.cuda.stream(stream):
            return method(*args, **kw)
    return call


def _run(name: str, device: torch.device, *args) -> None:
    """The library's `name`, of no plan, on the device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, not on {device}")
    with torch.cuda.device(device):
        _abi.check(getattr(_abi.lib(), name)(*args, _stream_handle(device, None)), name)


class ExpertWeights4:
    """Expert weights [experts, rows, in_features] in 4 bits, packed for expert_linear4: made by
    pack_experts4 or quantize_experts4.  packed: the buffer (uint8); one that was saved may take its
    place, in weights of the same sizes, format and group."""

    def __init__(self, experts: int, rows: int, in_features: int, format: str, group: int,
                 device: torch.device):
        if format not in _abi.WEIGHTS4:
            raise ValueError(f"format must be one of {tuple(_abi.WEIGHTS4)}")
        self.format, self.group = format, group
        self._cfg = _abi.Weights4Config(experts, rows, in_features, _abi.WEIGHTS4[format], group)
        self.cfg = ctypes.byref(self._cfg)
        size = _abi.lib().moe_weights4_bytes(self.cfg)
        if size == 0:
            raise ValueError(f"{format} weights of {experts} x {rows} x {in_features} in groups of "
                             f"{group} are not supported")
        self.packed = torch.empty(size, dtype=torch.uint8, device=device)
        self.device, self._size = self.packed.device, (size,)

    experts = property(lambda self: self._cfg.experts)
    rows = property(lambda self: self._cfg.rows)
    in_features = property(lambda self: self._cfg.in_features)

    def check(self, device: torch.device) -> None:
        """The library reads packed as long as the sizes say."""
        _need(self.packed, self._size, (torch.uint8,), "packed", device)

    def values(self, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
        """moe_weights4_unpack: the values that the weights stand for, [experts, rows,
        in_features] of dtype (float32 or bf16)."""
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the weights on {self.device}")
        return _values4(self, dtype, stream=stream)


@_on_stream
def _values4(w4: ExpertWeights4, dtype: torch.dtype) -> torch.Tensor:
    code = _out_code(dtype, "dtype")
    w4.check(w4.device)
    w = torch.empty((w4.experts, w4.rows, w4.in_features), dtype=dtype, device=w4.device)
    _run("moe_weights4_unpack", w4.device, w4.cfg,
         w4.packed.data_ptr(), w.data_ptr(), code)
    return w


@_on_stream
def pack_experts4(codes: torch.Tensor, scales: torch.Tensor, format: str = "int4",
                  group: int = 128) -> ExpertWeights4:
    """moe_weights4_pack: codes [experts, rows, in / 2] uint8 (weight 2j in the lower nibble of byte
    j) and scales [experts, rows, ceil(in / group)] as a checkpoint holds them -> packed weights.

    format "int4": scale * (code - 8), bf16 scales, groups of 32, 64 or 128; "e2m1": 2^(scale - 127)
    times the OCP E2M1 value, uint8 (E8M0) scales, groups of 32."""
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    if codes.dim() != 3:
        raise ValueError(f"codes has shape {tuple(codes.shape)}, expected [experts, rows, in / 2]")
    dev = codes.device
    E, Z, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    _need(codes, (E, Z, K // 2), (torch.uint8,), "codes", dev)
    w4 = ExpertWeights4(E, Z, K, format, group, dev)
    kinds = (torch.bfloat16,) if format == "int4" else (torch.uint8,)
    _need(scales, (E, Z, -(-K // group)), kinds, "scales", dev)
    _run("moe_weights4_pack", dev, w4.cfg, codes.data_ptr(),
         scales.data_ptr(), w4.packed.data_ptr())
    return w4


@_on_stream
def quantize_experts4(w: torch.Tensor, format: str = "int4", group: int = 128) -> ExpertWeights4:
    """moe_weights4_quantize: bf16 weights [experts, rows, in] -> packed weights.

    "int4": scale = max |w| / 7 of the group, rounded to bf16; "e2m1" (group 32): the smallest power
    of two with max |w| <= 6 * scale.  Codes are rounded to nearest even."""
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    if w.dim() != 3:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected [experts, rows, in]")
    _need(w, tuple(w.shape), _BF16, "w", w.device)
    w4 = ExpertWeights4(*w.shape, format, group, w.device)
    _run("moe_weights4_quantize", w.device, w4.cfg, w.data_ptr(),
         w4.packed.data_ptr())
    return w4


class Plan:
    """Owns one moe_plan (host) and, once routed, its device workspace tensor."""

    def __init__(self, num_tokens: int, hidden: int, num_experts: int, top_k: int,
                 num_ranks: int, ranks_per_node: int | None = None, node_dedup: bool = False,
                 load_aware_forwarders: bool = False, band_tokens: int = 0):
        G = num_ranks if ranks_per_node is None else ranks_per_node
        flags = (_abi.FLAG_NODE_DEDUP if node_dedup else 0) | \
            (_abi.FLAG_LOAD_AWARE_FORWARDERS if load_aware_forwarders else 0)
        self.cfg = _abi.MoeConfig(num_tokens, hidden, num_experts, top_k, num_ranks, G, flags,
                                  band_tokens)
        self._lib = _abi.lib()
        h = ctypes.c_void_p()
        _abi.check(self._lib.moe_plan_create(ctypes.byref(self.cfg), ctypes.byref(h)),
                   "moe_plan_create")
        self._h = h
        self.T, self.H, self.E, self.k = num_tokens, hidden, num_experts, top_k
        self.R, self.G, self.N = num_ranks, G, num_ranks // G
        self.node_dedup = node_dedup
        self.workspace_bytes = int(self._lib.moe_plan_workspace_bytes(h))
        self.recv_rows = int(self._lib.moe_plan_recv_rows(h))
        self.staging_rows_max = int(self._lib.moe_plan_staging_rows_max(h))
        self.scale_blocks = int(self._lib.moe_plan_scale_blocks(h))
        self.bands = int(self._lib.moe_plan_bands(h))
        # tokens per chunk of the chunked calls of a node-deduplicated plan
        self.chunk_tokens = {call: int(self._lib.moe_plan_chunk_tokens(h, i))
                             for i, call in enumerate(("dispatch", "dispatch_fp8", "combine_hier"))}
        self.workspace = None
        self.topk_idx = None
        self.device = None
        self._configs = {}   # of norm, norm_backward and expert_linear4, by what they say

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.moe_plan_destroy(h)
            self._h = None

    def _launch(self, name: str, device: torch.device, *args) -> None:
        """Calls the library's `name` on this plan and the device's current stream, with `device`
        current (a kernel is launched on the current device)."""
        if device.type != "cuda":
            raise ValueError(f"tensors must be on the GPU, not on {device}")
        # The raw handle: making a torch.cuda.Stream object takes 2 us, a sixth of a small call.
        stream = torch._C._cuda_getCurrentRawStream(device.index)
        fn = getattr(self._lib, name)
        if device.index == torch._C._cuda_getDevice():
            st = fn(self._h, *args, stream)
        else:
            with torch.cuda.device(device):
                st = fn(self._h, *args, stream)
        if st != _abi.OK:
            raise MoeError(st, name)

    # -- moe_route_plan
    def route(self, topk_idx: torch.Tensor, workspace: torch.Tensor | None = None, stream=None):
        dev = topk_idx.device
        _need(topk_idx, (self.T, self.k), (torch.int32,), "topk_idx", dev)
        if workspace is None:
            if self.workspace is None or self.workspace.device != dev:
                self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
            workspace = self.workspace
        elif workspace.numel() * workspace.element_size() < self.workspace_bytes:
            raise ValueError("workspace too small")
        self.workspace, self.topk_idx, self.device = workspace, topk_idx, dev
        _abi.check(self._lib.moe_route_plan(self._h, _ptr(topk_idx), _ptr(workspace),
                                            _stream_handle(dev, stream)), "moe_route_plan")
        return self

    # -- moe_route_plan_static
    def route_static(self, topk_idx: torch.Tensor, stream=None):
        """moe_route_plan_static: the route plan on the library's per-device
        static workspace; allocates nothing.  Plans routed this way on one GPU
        share that workspace: the last one routed is the one that holds it."""
        dev = topk_idx.device
        _need(topk_idx, (self.T, self.k), (torch.int32,), "topk_idx", dev)
        self.workspace, self.topk_idx, self.device = None, topk_idx, dev
        _abi.check(self._lib.moe_route_plan_static(self._h, _ptr(topk_idx),
                                                   _stream_handle(dev, stream)),
                   "moe_route_plan_static")
        return self

    # -- moe_pipeline
    def pipeline(self, topk_idx: torch.Tensor, x: torch.Tensor, topk_w: torch.Tensor,
                 recv: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None,
                 stream=None):
        """Route, dispatch and combine (identity expert) of every band in one launch.

        Returns (recv [T*k, H], out [T, H]); the plan is routed afterwards."""
        dev = topk_idx.device
        _need(topk_idx, (self.T, self.k), (torch.int32,), "topk_idx", dev)
        _need(x, (self.T, self.H), _BF16_LIKE, "x", dev)
        _need(topk_w, (self.T, self.k), (torch.float32,), "topk_w", dev)
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        if recv is None:
            recv = torch.empty((self.recv_rows, self.H), dtype=x.dtype, device=dev)
        _need(recv, (self.recv_rows, self.H), _BF16_LIKE, "recv", dev)
        if out is None:
            out = torch.empty((self.T, self.H), dtype=out_dtype, device=dev)
        _need(out, (self.T, self.H), (out_dtype,), "out", dev)
        if workspace is None:
            if self.workspace is None or self.workspace.device != dev:
                self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
            workspace = self.workspace
        elif workspace.numel() * workspace.element_size() < self.workspace_bytes:
            raise ValueError("workspace too small")
        self.workspace, self.topk_idx, self.device = workspace, topk_idx, dev
        code = _abi.OUT_F32 if out_dtype == torch.float32 else _abi.OUT_BF16
        _abi.check(self._lib.moe_pipeline(self._h, _ptr(topk_idx), _ptr(workspace), _ptr(x),
                                          _ptr(recv), _ptr(topk_w), _ptr(out), code,
                                          _stream_handle(dev, stream)), "moe_pipeline")
        return recv, out

    # -- moe_dispatch
    def dispatch(self, x: torch.Tensor, recv: torch.Tensor | None = None,
                 staging: torch.Tensor | None = None, stream=None):
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "dispatch")
        _need(x, (self.T, self.H), _BF16_LIKE, "x", dev)
        if recv is None:
            recv = torch.empty((self.recv_rows, self.H), dtype=x.dtype, device=dev)
        _need(recv, (self.recv_rows, self.H), _BF16_LIKE, "recv", dev)
        if self.node_dedup:
            if staging is None:
                staging = torch.empty((self.staging_rows_max, self.H), dtype=x.dtype, device=dev)
            _need(staging, (self.staging_rows_max, self.H), _BF16_LIKE, "staging", dev)
        _abi.check(self._lib.moe_dispatch(self._h, _ptr(x), _ptr(recv), _ptr(staging),
                                          _stream_handle(dev, stream)), "moe_dispatch")
        return recv, staging

    # -- moe_combine
    def combine(self, y: torch.Tensor, topk_w: torch.Tensor, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "combine")
        _need(y, (self.recv_rows, self.H), _BF16_LIKE, "y", dev)
        _need(topk_w, (self.T, self.k), (torch.float32,), "topk_w", dev)
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        if out is None:
            out = torch.empty((self.T, self.H), dtype=out_dtype, device=dev)
        _need(out, (self.T, self.H), (out_dtype,), "out", dev)
        code = _abi.OUT_F32 if out_dtype == torch.float32 else _abi.OUT_BF16
        _abi.check(self._lib.moe_combine(self._h, _ptr(y), _ptr(topk_w), _ptr(out), code,
                                         _stream_handle(dev, stream)), "moe_combine")
        return out

    # -- moe_combine_hier
    def combine_hier(self, y: torch.Tensor, topk_w: torch.Tensor,
                     partials: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """Two-hop combine of a node-deduplicated plan (fp32 partial per staging row)."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "combine_hier")
        _need(y, (self.recv_rows, self.H), _BF16_LIKE, "y", dev)
        _need(topk_w, (self.T, self.k), (torch.float32,), "topk_w", dev)
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        if partials is None:
            partials = torch.empty((self.staging_rows_max, self.H), dtype=torch.float32, device=dev)
        _need(partials, (self.staging_rows_max, self.H), (torch.float32,), "partials", dev)
        if out is None:
            out = torch.empty((self.T, self.H), dtype=out_dtype, device=dev)
        _need(out, (self.T, self.H), (out_dtype,), "out", dev)
        code = _abi.OUT_F32 if out_dtype == torch.float32 else _abi.OUT_BF16
        _abi.check(self._lib.moe_combine_hier(self._h, _ptr(y), _ptr(topk_w), _ptr(partials),
                                              _ptr(out), code, _stream_handle(dev, stream)),
                   "moe_combine_hier")
        return out

    # -- moe_dispatch_fp8
    def dispatch_fp8(self, x: torch.Tensor, recv8: torch.Tensor | None = None,
                     recv_scale: torch.Tensor | None = None, staging8: torch.Tensor | None = None,
                     staging_scale: torch.Tensor | None = None, stream=None):
        """fp8 payload: returns (codes uint8 [T*k, H], block scales float32 [T*k, nb]).

        With node deduplication the codes and scales pass through staging rows
        (staging8 [staging_rows_max, H] uint8, staging_scale [.., nb] float32)."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "dispatch_fp8")
        _need(x, (self.T, self.H), _BF16_LIKE, "x", dev)
        if recv8 is None:
            recv8 = torch.empty((self.recv_rows, self.H), dtype=torch.uint8, device=dev)
        if recv_scale is None:
            recv_scale = torch.empty((self.recv_rows, self.scale_blocks), dtype=torch.float32,
                                     device=dev)
        _need(recv8, (self.recv_rows, self.H), (torch.uint8,), "recv8", dev)
        _need(recv_scale, (self.recv_rows, self.scale_blocks), (torch.float32,), "recv_scale", dev)
        if self.node_dedup:
            D = self.staging_rows_max
            if staging8 is None:
                staging8 = torch.empty((D, self.H), dtype=torch.uint8, device=dev)
            if staging_scale is None:
                staging_scale = torch.empty((D, self.scale_blocks), dtype=torch.float32, device=dev)
            _need(staging8, (D, self.H), (torch.uint8,), "staging8", dev)
            _need(staging_scale, (D, self.scale_blocks), (torch.float32,), "staging_scale", dev)
        _abi.check(self._lib.moe_dispatch_fp8(self._h, _ptr(x), _ptr(recv8), _ptr(recv_scale),
                                              _ptr(staging8), _ptr(staging_scale),
                                              _stream_handle(dev, stream)), "moe_dispatch_fp8")
        return recv8, recv_scale

    # -- moe_combine_fp8
    def combine_fp8(self, y8: torch.Tensor, y_scale: torch.Tensor, topk_w: torch.Tensor,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                    stream=None) -> torch.Tensor:
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "combine_fp8")
        _need(y8, (self.recv_rows, self.H), (torch.uint8,), "y8", dev)
        _need(y_scale, (self.recv_rows, self.scale_blocks), (torch.float32,), "y_scale", dev)
        _need(topk_w, (self.T, self.k), (torch.float32,), "topk_w", dev)
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        if out is None:
            out = torch.empty((self.T, self.H), dtype=out_dtype, device=dev)
        _need(out, (self.T, self.H), (out_dtype,), "out", dev)
        code = _abi.OUT_F32 if out_dtype == torch.float32 else _abi.OUT_BF16
        _abi.check(self._lib.moe_combine_fp8(self._h, _ptr(y8), _ptr(y_scale), _ptr(topk_w),
                                             _ptr(out), code, _stream_handle(dev, stream)),
                   "moe_combine_fp8")
        return out

    # -- moe_router
    def _router_config(self, score: str, renormalise: bool, nodes_per_token: int, scale: float,
                       key: str = "logit"):
        if score not in _abi.SCORE:
            raise ValueError(f"score must be one of {tuple(_abi.SCORE)}")
        if key not in _abi.ROUTER_KEY:
            raise ValueError(f"key must be one of {tuple(_abi.ROUTER_KEY)}")
        return ctypes.byref(_abi.RouterConfig(_abi.SCORE[score], bool(renormalise), nodes_per_token,
                                              scale, _abi.ROUTER_KEY[key]))

    @_on_stream
    def router(self, logits: torch.Tensor, bias: torch.Tensor | None = None,
               score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
               nodes_per_token: int = 0, topk_idx: torch.Tensor | None = None,
               topk_w: torch.Tensor | None = None, key: str = "logit"):
        """Gate logits [T, E] (float32 or bf16) -> (topk_idx int32 [T, k], topk_w float32 [T, k]).

        The k experts of the largest key + bias (bias: float32 [E], for the choice only), in
        descending order, ties to the lower id; nodes_per_token m > 0 allows the experts of the
        token's m best nodes only, by the sum of a node's two largest.  key: "logit", or "score"
        for the softmax or sigmoid of the logits; a bias belongs to the one it was adjusted for
        (DeepSeek-V3's routing: score="sigmoid", key="score").  Weights: scale * softmax or sigmoid
        of the logits, over the sum of the selected ones with renormalise.  The plan need not be
        routed."""
        dev = logits.device
        _need(logits, (self.T, self.E), (torch.float32, torch.bfloat16), "logits", dev)
        if bias is not None:
            _need(bias, (self.E,), _F32, "bias", dev)
        cfg = self._router_config(score, renormalise, nodes_per_token, scale, key)
        if topk_idx is not None or topk_w is not None:
            _apart((topk_idx, topk_w), (logits, bias))
        topk_idx = _out(topk_idx, (self.T, self.k), torch.int32, "topk_idx", dev)
        topk_w = _out(topk_w, (self.T, self.k), torch.float32, "topk_w", dev)
        self._launch("moe_router", dev, cfg, logits.data_ptr(), _OUT_CODE[logits.dtype],
                     _addr(bias), topk_idx.data_ptr(), topk_w.data_ptr())
        return topk_idx, topk_w

    # -- moe_router_backward
    @_on_stream
    def router_backward(self, logits: torch.Tensor, topk_idx: torch.Tensor, grad_w: torch.Tensor,
                        score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                        grad_logits: torch.Tensor | None = None) -> torch.Tensor:
        """Gradient of the weights with respect to the logits (the choice fixed): [T, E], every
        entry written, of the logits' dtype."""
        dev = logits.device
        _need(logits, (self.T, self.E), (torch.float32, torch.bfloat16), "logits", dev)
        _need(topk_idx, (self.T, self.k), (torch.int32,), "topk_idx", dev)
        _need(grad_w, (self.T, self.k), _F32, "grad_w", dev)
        cfg = self._router_config(score, renormalise, 0, scale)
        if grad_logits is not None:
            _apart((grad_logits,), (logits, topk_idx, grad_w))
        grad_logits = _out(grad_logits, (self.T, self.E), logits.dtype, "grad_logits", dev)
        self._launch("moe_router_backward", dev, cfg, logits.data_ptr(),
                     _OUT_CODE[logits.dtype], topk_idx.data_ptr(), grad_w.data_ptr(),
                     grad_logits.data_ptr())
        return grad_logits

    # -- moe_dispatch_backward
    @_on_stream
    def dispatch_backward(self, grad_recv: torch.Tensor, grad_x: torch.Tensor | None = None,
                          out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """Gradient of dispatch: grad_x[t] = sum_j grad_recv[slot_of[t, j]], [T, H]."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "dispatch_backward")
        _need(grad_recv, (self.recv_rows, self.H), _BF16_LIKE, "grad_recv", dev)
        code = _out_code(out_dtype, "out_dtype")
        if grad_x is not None:
            _apart((grad_x,), (grad_recv,))
        grad_x = _out(grad_x, (self.T, self.H), out_dtype, "grad_x", dev)
        self._launch("moe_dispatch_backward", dev, grad_recv.data_ptr(), grad_x.data_ptr(),
                     code)
        return grad_x

    # -- moe_combine_backward
    @_on_stream
    def combine_backward(self, grad_out: torch.Tensor, y: torch.Tensor, topk_w: torch.Tensor,
                         grad_y: torch.Tensor | None = None, grad_w: torch.Tensor | None = None):
        """Gradient of combine and combine_hier: returns (grad_y [T*k, H] bf16 in the receive
        layout, grad_w [T, k] float32); grad_out: [T, H] bf16 or float32."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "combine_backward")
        _need(grad_out, (self.T, self.H), (torch.float32, torch.bfloat16), "grad_out", dev)
        _need(y, (self.recv_rows, self.H), _BF16_LIKE, "y", dev)
        _need(topk_w, (self.T, self.k), _F32, "topk_w", dev)
        if grad_y is not None or grad_w is not None:
            _apart((grad_y, grad_w), (grad_out, y, topk_w))
        grad_y = _out(grad_y, (self.recv_rows, self.H), torch.bfloat16, "grad_y", dev)
        grad_w = _out(grad_w, (self.T, self.k), torch.float32, "grad_w", dev)
        self._launch("moe_combine_backward", dev, grad_out.data_ptr(),
                     _OUT_CODE[grad_out.dtype], y.data_ptr(), topk_w.data_ptr(), grad_y.data_ptr(),
                     grad_w.data_ptr())
        return grad_y, grad_w

    # -- moe_expert_linear
    def _expert_config(self, w: torch.Tensor, activation: str):
        """(config, K, N, Z) of a product with weights w [E, Z, K]."""
        if activation not in _abi.ACTIVATION:
            raise ValueError(f"activation must be one of {tuple(_abi.ACTIVATION)}")
        if not isinstance(w, torch.Tensor):
            raise TypeError("w must be a torch.Tensor")
        if w.dim() != 3:
            raise ValueError(f"w has shape {tuple(w.shape)}, expected [experts, out, in]")
        Z, K = w.shape[1], w.shape[2]
        N = Z
        if activation in _abi.GATED:
            if Z % 2:
                raise ValueError("a gated activation needs an even number of weight rows")
            N = Z // 2
        _need(w, (self.E, Z, K), _BF16, "w", self.device)
        return ctypes.byref(_abi.ExpertConfig(K, N, _abi.ACTIVATION[activation])), K, N, Z

    @_on_stream
    def expert_linear(self, x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
                      residual: torch.Tensor | None = None, activation: str = "none",
                      save_pre: bool = False, y: torch.Tensor | None = None,
                      pre: torch.Tensor | None = None):
        """Every expert's product on its rows of the receive layout: returns (y, pre).

        y[r] = act(x[r] . w[e]^T + bias[e]) + residual[r] for each receive row r of expert e;
        x [T*k, K], w [E, Z, K], residual and y [T*k, N] bf16, bias [E, Z] float32; Z = 2N (gate
        rows, then up rows) with "swiglu" and "geglu", else N.  pre: the product before the
        activation, [T*k, Z] bf16, with save_pre (or a tensor to write), else None.  K and N are
        multiples of 8."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "expert_linear")
        cfg, K, N, Z = self._expert_config(w, activation)
        rows = self.recv_rows
        _need(x, (rows, K), _BF16, "x", dev)
        if bias is not None:
            _need(bias, (self.E, Z), _F32, "bias", dev)
        if residual is not None:
            _need(residual, (rows, N), _BF16, "residual", dev)
        if y is not None or pre is not None:
            _apart((y, pre), (x, w, bias, residual))
        y = _out(y, (rows, N), torch.bfloat16, "y", dev)
        if save_pre or pre is not None:
            pre = _out(pre, (rows, Z), torch.bfloat16, "pre", dev)
        self._launch("moe_expert_linear", dev, cfg, x.data_ptr(), w.data_ptr(), _addr(bias),
                     _addr(residual), y.data_ptr(), _addr(pre))
        return y, pre

    # -- moe_expert_linear_backward
    @_on_stream
    def expert_linear_backward(self, grad_y: torch.Tensor, x: torch.Tensor | None, w: torch.Tensor,
                               pre: torch.Tensor | None = None, activation: str = "none",
                               bias_grad: bool = False, x_grad: bool = True, w_grad: bool = True,
                               grad_w_dtype: torch.dtype = torch.bfloat16,
                               grad_x: torch.Tensor | None = None,
                               grad_w: torch.Tensor | None = None,
                               grad_bias: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None):
        """Gradient of expert_linear: returns (grad_x [T*k, K] bf16, grad_w [E, Z, K] of
        grad_w_dtype, grad_bias [E, Z] float32), None for one that is not wanted.

        pre: what expert_linear stored, needed with an activation.  x_grad, w_grad, bias_grad say
        which are wanted; grad_x, grad_w, grad_bias: tensors to write them to.  x is read for grad_w
        only and may be None without it; w also says the sizes.  The gradient of the residual is
        grad_y."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "expert_linear_backward")
        cfg, K, N, Z = self._expert_config(w, activation)
        rows = self.recv_rows
        _need(grad_y, (rows, N), _BF16, "grad_y", dev)
        if w_grad or x is not None:
            _need(x, (rows, K), _BF16, "x", dev)
        if activation != "none":
            if pre is None:
                raise ValueError("pre is needed with an activation")
            _need(pre, (rows, Z), _BF16, "pre", dev)
        else:
            pre = None
        code = _out_code(grad_w_dtype, "grad_w_dtype")
        need = self._lib.moe_expert_backward_workspace_bytes(self._h, cfg)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        else:
            _need(workspace, getattr(workspace, "shape", ()), (getattr(workspace, "dtype", None),),
                  "workspace", dev)
            if workspace.numel() * workspace.element_size() < need:
                raise ValueError("workspace too small")
            _apart((workspace,), (grad_y, x, w, pre))
        given = tuple(t for t, wanted in ((grad_x, x_grad), (grad_w, w_grad), (grad_bias, bias_grad))
                      if wanted and t is not None)
        if given:
            _apart(given, (grad_y, x, w, pre, workspace))
        grad_x = _out(grad_x, (rows, K), torch.bfloat16, "grad_x", dev) if x_grad else None
        grad_w = _out(grad_w, (self.E, Z, K), grad_w_dtype, "grad_w", dev) if w_grad else None
        grad_bias = _out(grad_bias, (self.E, Z), torch.float32, "grad_bias", dev) if bias_grad else None
        self._launch("moe_expert_linear_backward", dev, cfg, grad_y.data_ptr(), _addr(x),
                     w.data_ptr(), _addr(pre), _addr(grad_x), _addr(grad_w), code, _addr(grad_bias),
                     workspace.data_ptr())
        return grad_x, grad_w, grad_bias

    # -- moe_expert_linear4
    @_on_stream
    def expert_linear4(self, x: torch.Tensor, w4: ExpertWeights4, bias: torch.Tensor | None = None,
                       residual: torch.Tensor | None = None, activation: str = "none",
                       y: torch.Tensor | None = None) -> torch.Tensor:
        """expert_linear with 4-bit weights, for serving (no gradient): returns y [T*k, N] bf16.

        w4: what pack_experts4 or quantize_experts4 made of weights [E, Z, K]; Z = 2N (gate rows,
        then up rows) with "swiglu" and "geglu", else N.  x [T*k, K], residual [T*k, N] bf16, bias
        [E, Z] float32."""
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "expert_linear4")
        if activation not in _abi.ACTIVATION:
            raise ValueError(f"activation must be one of {tuple(_abi.ACTIVATION)}")
        if not isinstance(w4, ExpertWeights4):
            raise TypeError("w4 must be ExpertWeights4")
        if w4.experts != self.E:
            raise ValueError(f"w4 has {w4.experts} experts, expected {self.E}")
        K, Z = w4.in_features, w4.rows
        N = Z
        if activation in _abi.GATED:
            if Z % 16:
                raise ValueError("a gated activation needs halves of a multiple of 8 weight rows")
            N = Z // 2
        rows = self.recv_rows
        w4.check(dev)
        _need(x, (rows, K), _BF16, "x", dev)
        if bias is not None:
            _need(bias, (self.E, Z), _F32, "bias", dev)
        if residual is not None:
            _need(residual, (rows, N), _BF16, "residual", dev)
        if y is not None:
            _apart((y,), (x, w4.packed, bias, residual))
        y = _out(y, (rows, N), torch.bfloat16, "y", dev)
        cfg = self._configs.get((K, N, activation))
        if cfg is None:
            cfg = ctypes.byref(_abi.ExpertConfig(K, N, _abi.ACTIVATION[activation]))
            self._configs[(K, N, activation)] = cfg
        self._launch("moe_expert_linear4", dev, cfg, w4.cfg, x.data_ptr(), w4.packed.data_ptr(),
                     _addr(bias), _addr(residual), y.data_ptr())
        return y

    # -- moe_norm
    def _norm_config(self, kind: str, eps: float, x: torch.Tensor, y_code: int):
        """(config, bytes of norm_backward's workspace)"""
        at = (kind, eps, x.dtype, y_code)
        if at not in self._configs:     # making one takes 1 us, asking for the bytes another
            if kind not in _abi.NORM:
                raise ValueError(f"kind must be one of {tuple(_abi.NORM)}")
            cfg = ctypes.byref(_abi.NormConfig(_abi.NORM[kind], eps, _OUT_CODE[x.dtype], y_code))
            self._configs[at] = cfg, self._lib.moe_norm_backward_workspace_bytes(self._h, cfg)
        return self._configs[at]

    @_on_stream
    def norm(self, x: torch.Tensor, gamma: torch.Tensor | None = None,
             beta: torch.Tensor | None = None, residual: torch.Tensor | None = None,
             kind: str = "layer", eps: float = 1e-5, out_dtype: torch.dtype = torch.bfloat16,
             save_stats: bool = False, y: torch.Tensor | None = None,
             total: torch.Tensor | None = None, stats: torch.Tensor | None = None):
        """Norm of the residual stream's rows: returns (y, total, stats).

        total = x + residual, rounded to x's dtype (None without a residual: x is what is normed);
        y = (total - mean) * rstd * gamma + beta, [T, H] of out_dtype; kind: "layer", or "rms" for
        mean = 0.  x, residual: [T, H] float32 or bf16, of one dtype; gamma, beta: [H] float32 (None:
        ones, zeros).  stats: [T, 2] float32 (mean, rstd) for the gradient, with save_stats (or a
        tensor to write), else None.  The plan need not be routed."""
        dev = x.device
        _need(x, (self.T, self.H), (torch.float32, torch.bfloat16), "x", dev)
        for t, name in ((gamma, "gamma"), (beta, "beta")):
            if t is not None:
                _need(t, (self.H,), _F32, name, dev)
        if residual is not None:
            _need(residual, (self.T, self.H), (x.dtype,), "residual", dev)
        elif total is not None:
            raise ValueError("total is written with a residual only")
        cfg, _ = self._norm_config(kind, eps, x, _out_code(out_dtype, "out_dtype"))
        if y is not None or total is not None or stats is not None:
            _apart((y, total, stats), (x, gamma, beta, residual))
        y = _out(y, (self.T, self.H), out_dtype, "y", dev)
        if residual is not None:
            total = _out(total, (self.T, self.H), x.dtype, "total", dev)
        if save_stats or stats is not None:
            stats = _out(stats, (self.T, 2), torch.float32, "stats", dev)
        self._launch("moe_norm", dev, cfg, x.data_ptr(), _addr(residual), _addr(gamma), _addr(beta),
                     y.data_ptr(), _addr(total), _addr(stats))
        return y, total, stats

    # -- moe_norm_backward
    @_on_stream
    def norm_backward(self, grad_y: torch.Tensor, total: torch.Tensor, stats: torch.Tensor,
                      gamma: torch.Tensor | None = None, grad_total: torch.Tensor | None = None,
                      kind: str = "layer", x_grad: bool = True, gamma_grad: bool = True,
                      beta_grad: bool = True, grad_x: torch.Tensor | None = None,
                      grad_gamma: torch.Tensor | None = None,
                      grad_beta: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
        """Gradient of norm: returns (grad_x [T, H] of total's dtype, grad_gamma and grad_beta [H]
        float32), None for one that is not wanted.

        total: what was normed (norm's second output, or its x without a residual); stats: as norm
        stored them; grad_y: [T, H] float32 or bf16; grad_total: [T, H] of total's dtype, the
        gradient that reaches total by other ways, added to grad_x.  grad_x is the gradient of x
        and of the residual.  x_grad, gamma_grad, beta_grad say which are wanted; grad_x,
        grad_gamma, grad_beta: tensors to write them to."""
        dev = total.device
        _need(total, (self.T, self.H), (torch.float32, torch.bfloat16), "total", dev)
        _need(grad_y, (self.T, self.H), (torch.float32, torch.bfloat16), "grad_y", dev)
        _need(stats, (self.T, 2), _F32, "stats", dev)
        if gamma is not None:
            _need(gamma, (self.H,), _F32, "gamma", dev)
        if grad_total is not None:
            _need(grad_total, (self.T, self.H), (total.dtype,), "grad_total", dev)
        cfg, need = self._norm_config(kind, 0.0, total, _OUT_CODE[grad_y.dtype])
        inputs = (grad_y, total, stats, gamma, grad_total)
        if workspace is not None:
            _need(workspace, getattr(workspace, "shape", ()), (getattr(workspace, "dtype", None),),
                  "workspace", dev)
            if workspace.numel() * workspace.element_size() < need:
                raise ValueError("workspace too small")
            _apart((workspace,), inputs)
        elif need and (gamma_grad or beta_grad):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        given = tuple(t for t, wanted in ((grad_x, x_grad), (grad_gamma, gamma_grad),
                                          (grad_beta, beta_grad)) if wanted and t is not None)
        if given:
            _apart(given, (*inputs, workspace))
        grad_x = _out(grad_x, (self.T, self.H), total.dtype, "grad_x", dev) if x_grad else None
        grad_gamma = _vector(grad_gamma, self.H, "grad_gamma", dev) if gamma_grad else None
        grad_beta = _vector(grad_beta, self.H, "grad_beta", dev) if beta_grad else None
        self._launch("moe_norm_backward", dev, cfg, grad_y.data_ptr(), total.data_ptr(),
                     stats.data_ptr(), _addr(gamma), _addr(grad_total), _addr(grad_x),
                     _addr(grad_gamma), _addr(grad_beta), _addr(workspace))
        return grad_x, grad_gamma, grad_beta

    # -- moe_plan_timing / moe_plan_timing_read
    def timing(self, capacity: int) -> None:
        """Time each kernel this plan's calls launch (up to `capacity` launches;
        0 stops).  Needs the plan's device to be current."""
        _abi.check(self._lib.moe_plan_timing(self._h, int(capacity)), "moe_plan_timing")
        self._timing_cap = int(capacity)

    def timing_read(self) -> list[tuple[str, float, float]]:
        """(kernel name, start in ms after the first launch's start, duration in ms) of
        each timed launch since the last read, in launch order."""
        cap = getattr(self, "_timing_cap", 0)
        ids = (ctypes.c_int32 * max(cap, 1))()
        start = (ctypes.c_float * max(cap, 1))()
        ms = (ctypes.c_float * max(cap, 1))()
        n = ctypes.c_int32()
        _abi.check(self._lib.moe_plan_timing_read(self._h, ids, start, ms, cap, ctypes.byref(n)),
                   "moe_plan_timing_read")
        return [(_abi.kernel_name(ids[i]), float(start[i]), float(ms[i]))
                for i in range(min(n.value, cap))]

    # -- moe_plan_read
    def read(self, item: str, stream=None) -> np.ndarray:
        nb = self.bands
        n = {"status": 1, "num_staged": 1, "counts": nb * self.E,
             "expert_offsets": nb * (self.E + 1), "rank_offsets": nb * (self.R + 1),
             "slot_of": self.T * self.k, "row_src": self.T * self.k,
             "stage_offsets": self.R + 1, "stage_of": self.T * self.k,
             "stage_src": self.staging_rows_max, "send_rows": self.R * self.R,
             "send_copies": self.R * self.R, "node_copies": self.R * self.N,
             "forwarders": self.R * self.N}[item]
        buf = np.zeros(max(n, 1), dtype=np.int32)
        dev = self.device
        if dev is None:
            raise MoeError(_abi.ERR_PLAN_NOT_ROUTED, "read")
        _abi.check(self._lib.moe_plan_read(self._h, _abi.ITEM[item],
                                           buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                           _stream_handle(dev, stream)), f"moe_plan_read({item})")
        return buf[:n]

    def status(self) -> int:
        return int(self.read("status")[0])


def route_plan(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, hidden: int,
               ranks_per_node: int | None = None, node_dedup: bool = False,
               load_aware_forwarders: bool = False, workspace: torch.Tensor | None = None,
               stream=None) -> Plan:
    """moe_plan_create + moe_route_plan for a [T, k] int32 routing on the GPU."""
    T, k = topk_idx.shape
    plan = Plan(T, hidden, num_experts, k, num_ranks, ranks_per_node, node_dedup,
                load_aware_forwarders)
    return plan.route(topk_idx, workspace, stream)


def dispatch(plan: Plan, x: torch.Tensor, recv=None, staging=None, stream=None):
    """moe_dispatch: returns (recv [T*k, H], staging or None)."""
    return plan.dispatch(x, recv, staging, stream)


def combine(plan: Plan, y: torch.Tensor, topk_w: torch.Tensor, out=None,
            out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_combine: returns out [T, H] (bf16 or float32)."""
    return plan.combine(y, topk_w, out, out_dtype, stream)


def dispatch_fp8(plan: Plan, x: torch.Tensor, recv8=None, recv_scale=None, staging8=None,
                 staging_scale=None, stream=None):
    """moe_dispatch_fp8: returns (codes [T*k, H] uint8, block scales [T*k, nb] float32)."""
    return plan.dispatch_fp8(x, recv8, recv_scale, staging8, staging_scale, stream)


def combine_fp8(plan: Plan, y8: torch.Tensor, y_scale: torch.Tensor, topk_w: torch.Tensor,
                out=None, out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_combine_fp8: returns out [T, H] (bf16 or float32)."""
    return plan.combine_fp8(y8, y_scale, topk_w, out, out_dtype, stream)


def combine_hier(plan: Plan, y: torch.Tensor, topk_w: torch.Tensor, partials=None, out=None,
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_combine_hier: two-hop combine of a node-deduplicated plan."""
    return plan.combine_hier(y, topk_w, partials, out, out_dtype, stream)


def pipeline(plan: Plan, topk_idx: torch.Tensor, x: torch.Tensor, topk_w: torch.Tensor,
             recv=None, out=None, out_dtype: torch.dtype = torch.bfloat16, stream=None):
    """moe_pipeline: returns (recv [T*k, H], out [T, H])."""
    return plan.pipeline(topk_idx, x, topk_w, recv, out, out_dtype, stream=stream)


def router(plan: Plan, logits: torch.Tensor, bias=None, score: str = "softmax",
           renormalise: bool = True, scale: float = 1.0, nodes_per_token: int = 0, topk_idx=None,
           topk_w=None, stream=None, key: str = "logit"):
    """moe_router: returns (topk_idx [T, k] int32, topk_w [T, k] float32)."""
    return plan.router(logits, bias, score, renormalise, scale, nodes_per_token, topk_idx, topk_w,
                       key, stream=stream)


def router_backward(plan: Plan, logits: torch.Tensor, topk_idx: torch.Tensor, grad_w: torch.Tensor,
                    score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                    grad_logits=None, stream=None) -> torch.Tensor:
    """moe_router_backward: returns grad_logits [T, E]."""
    return plan.router_backward(logits, topk_idx, grad_w, score, renormalise, scale, grad_logits,
                                stream=stream)


def dispatch_backward(plan: Plan, grad_recv: torch.Tensor, grad_x=None,
                      out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_dispatch_backward: returns grad_x [T, H] (bf16 or float32)."""
    return plan.dispatch_backward(grad_recv, grad_x, out_dtype, stream=stream)


def combine_backward(plan: Plan, grad_out: torch.Tensor, y: torch.Tensor, topk_w: torch.Tensor,
                     grad_y=None, grad_w=None, stream=None):
    """moe_combine_backward: returns (grad_y [T*k, H] bf16, grad_w [T, k] float32)."""
    return plan.combine_backward(grad_out, y, topk_w, grad_y, grad_w, stream=stream)


def expert_linear(plan: Plan, x: torch.Tensor, w: torch.Tensor, bias=None, residual=None,
                  activation: str = "none", save_pre: bool = False, y=None, pre=None, stream=None):
    """moe_expert_linear: returns (y [T*k, N] bf16, pre [T*k, Z] bf16 or None)."""
    return plan.expert_linear(x, w, bias, residual, activation, save_pre, y, pre,
                              stream=stream)


def expert_linear_backward(plan: Plan, grad_y: torch.Tensor, x: torch.Tensor | None, w: torch.Tensor,
                           pre=None, activation: str = "none", bias_grad: bool = False,
                           x_grad: bool = True, w_grad: bool = True,
                           grad_w_dtype: torch.dtype = torch.bfloat16, grad_x=None, grad_w=None,
                           grad_bias=None, workspace=None, stream=None):
    """moe_expert_linear_backward: returns (grad_x, grad_w, grad_bias), None where not wanted."""
    return plan.expert_linear_backward(grad_y, x, w, pre, activation, bias_grad, x_grad, w_grad,
                                       grad_w_dtype, grad_x, grad_w, grad_bias, workspace,
                                       stream=stream)


def expert_linear4(plan: Plan, x: torch.Tensor, w4: ExpertWeights4, bias=None, residual=None,
                   activation: str = "none", y=None, stream=None) -> torch.Tensor:
    """moe_expert_linear4: returns y [T*k, N] bf16."""
    return plan.expert_linear4(x, w4, bias, residual, activation, y, stream=stream)


def norm(plan: Plan, x: torch.Tensor, gamma=None, beta=None, residual=None, kind: str = "layer",
         eps: float = 1e-5, out_dtype: torch.dtype = torch.bfloat16, save_stats: bool = False, y=None,
         total=None, stats=None, stream=None):
    """moe_norm: returns (y [T, H], total [T, H] or None, stats [T, 2] float32 or None)."""
    return plan.norm(x, gamma, beta, residual, kind, eps, out_dtype, save_stats, y, total, stats,
                     stream=stream)


def norm_backward(plan: Plan, grad_y: torch.Tensor, total: torch.Tensor, stats: torch.Tensor,
                  gamma=None, grad_total=None, kind: str = "layer", x_grad: bool = True,
                  gamma_grad: bool = True, beta_grad: bool = True, grad_x=None, grad_gamma=None,
                  grad_beta=None, workspace=None, stream=None):
    """moe_norm_backward: returns (grad_x, grad_gamma, grad_beta), None where not wanted."""
    return plan.norm_backward(grad_y, total, stats, gamma, grad_total, kind, x_grad, gamma_grad,
                              beta_grad, grad_x, grad_gamma, grad_beta, workspace, stream=stream)
