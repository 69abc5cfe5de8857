"""ctypes declarations of the C ABI in include/moe_shuffle.h, include/moe_layer.h and
include/moe_block.h.

Loads the in-tree libmoeshuffle.so and fails loudly when it is missing: there
is no fallback of any kind.
"""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoeshuffle.so")

# moe_status
OK = 0
ERR_INVALID_ARGUMENT = 1
ERR_EXPERTS_LT_RANKS = 2
ERR_BAD_ROUTING = 3
ERR_PLAN_NOT_ROUTED = 4
ERR_HIP = 5
ERR_UNSUPPORTED = 6
ERR_PIPELINE_STALL = 7
ERR_STATIC_WORKSPACE = 8
STATIC_WORKSPACE_BYTES = 32 << 20

FLAG_NODE_DEDUP = 1
FLAG_LOAD_AWARE_FORWARDERS = 2
MAX_EXPERTS = 1024
MAX_TOPK = 16

OUT_BF16 = 0
OUT_F32 = 1

# moe_layer.h: moe_score, moe_router_key, moe_activation
SCORE = dict(softmax=0, sigmoid=1)
ROUTER_KEY = dict(logit=0, score=1)
ACTIVATION = dict(none=0, relu=1, silu=2, gelu=3, swiglu=4, geglu=5)
GATED = ("swiglu", "geglu")

# moe_block.h: moe_norm_kind, moe_weights4_format
NORM = dict(layer=0, rms=1)
WEIGHTS4 = dict(int4=0, e2m1=1)

# moe_item
ITEM = dict(status=0, counts=1, expert_offsets=2, rank_offsets=3, slot_of=4, row_src=5,
            num_staged=6, stage_offsets=7, stage_of=8, stage_src=9, send_rows=10,
            send_copies=11, node_copies=12, forwarders=13)


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("ranks_per_node", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("band_tokens", ctypes.c_int32),
    ]


class RouterConfig(ctypes.Structure):
    _fields_ = [
        ("score", ctypes.c_int32),
        ("renormalise", ctypes.c_int32),
        ("nodes_per_token", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("key", ctypes.c_int32),
    ]


class ExpertConfig(ctypes.Structure):
    _fields_ = [
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("activation", ctypes.c_int32),
    ]


class NormConfig(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("x_dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
    ]


class Weights4Config(ctypes.Structure):
    _fields_ = [
        ("experts", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("in_features", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("group", ctypes.c_int32),
    ]


# include/moe_shuffle.h
EXPORTS = (
    "moe_expert_partition", "moe_plan_create", "moe_plan_destroy", "moe_plan_workspace_bytes",
    "moe_plan_recv_rows", "moe_plan_staging_rows_max", "moe_route_plan", "moe_dispatch",
    "moe_combine", "moe_plan_read", "moe_status_str", "moe_plan_scale_blocks",
    "moe_dispatch_fp8", "moe_combine_fp8", "moe_combine_hier", "moe_plan_bands", "moe_pipeline",
    "moe_kernel_name", "moe_plan_timing", "moe_plan_timing_read", "moe_route_plan_static",
    "moe_plan_chunk_tokens",
)

# include/moe_layer.h
LAYER_EXPORTS = (
    "moe_router", "moe_router_backward", "moe_dispatch_backward", "moe_combine_backward",
    "moe_expert_linear", "moe_expert_backward_workspace_bytes", "moe_expert_linear_backward",
)

# include/moe_block.h
BLOCK_EXPORTS = (
    "moe_norm", "moe_norm_backward_workspace_bytes", "moe_norm_backward", "moe_weights4_bytes",
    "moe_weights4_pack", "moe_weights4_quantize", "moe_weights4_unpack", "moe_expert_linear4",
)

KERNEL_COUNT = 33  # moe_kernel and moe_layer_kernel
BLOCK_KERNELS = range(64, 69)  # moe_block_kernel


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m combine_shuffling_amd.build` "
            "(hipcc, gfx950). There is no fallback path.")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.moe_expert_partition.argtypes = [i32, i32, ctypes.POINTER(i32)]
    L.moe_expert_partition.restype = i32
    L.moe_plan_create.argtypes = [ctypes.POINTER(MoeConfig), ctypes.POINTER(vp)]
    L.moe_plan_create.restype = i32
    L.moe_plan_destroy.argtypes = [vp]
    L.moe_plan_destroy.restype = None
    L.moe_plan_workspace_bytes.argtypes = [vp]
    L.moe_plan_workspace_bytes.restype = sz
    L.moe_plan_recv_rows.argtypes = [vp]
    L.moe_plan_recv_rows.restype = i64
    L.moe_plan_staging_rows_max.argtypes = [vp]
    L.moe_plan_staging_rows_max.restype = i64
    L.moe_route_plan.argtypes = [vp, vp, vp, vp]
    L.moe_route_plan.restype = i32
    L.moe_dispatch.argtypes = [vp, vp, vp, vp, vp]
    L.moe_dispatch.restype = i32
    L.moe_combine.argtypes = [vp, vp, vp, vp, i32, vp]
    L.moe_combine.restype = i32
    L.moe_plan_read.argtypes = [vp, i32, vp, sz, vp]
    L.moe_plan_read.restype = i32
    L.moe_plan_scale_blocks.argtypes = [vp]
    L.moe_plan_scale_blocks.restype = i64
    L.moe_dispatch_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    L.moe_dispatch_fp8.restype = i32
    L.moe_combine_fp8.argtypes = [vp, vp, vp, vp, vp, i32, vp]
    L.moe_combine_fp8.restype = i32
    L.moe_combine_hier.argtypes = [vp, vp, vp, vp, vp, i32, vp]
    L.moe_combine_hier.restype = i32
    L.moe_plan_chunk_tokens.argtypes = [vp, i32]
    L.moe_plan_chunk_tokens.restype = i64
    L.moe_plan_bands.argtypes = [vp]
    L.moe_plan_bands.restype = i64
    L.moe_pipeline.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp]
    L.moe_pipeline.restype = i32
    L.moe_route_plan_static.argtypes = [vp, vp, vp]
    L.moe_route_plan_static.restype = i32
    L.moe_kernel_name.argtypes = [i32]
    L.moe_kernel_name.restype = ctypes.c_char_p
    L.moe_plan_timing.argtypes = [vp, i32]
    L.moe_plan_timing.restype = i32
    L.moe_plan_timing_read.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_float),
                                       ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(i32)]
    L.moe_plan_timing_read.restype = i32
    router, expert = ctypes.POINTER(RouterConfig), ctypes.POINTER(ExpertConfig)
    L.moe_router.argtypes = [vp, router, vp, i32, vp, vp, vp, vp]
    L.moe_router.restype = i32
    L.moe_router_backward.argtypes = [vp, router, vp, i32, vp, vp, vp, vp]
    L.moe_router_backward.restype = i32
    L.moe_dispatch_backward.argtypes = [vp, vp, vp, i32, vp]
    L.moe_dispatch_backward.restype = i32
    L.moe_combine_backward.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp]
    L.moe_combine_backward.restype = i32
    L.moe_expert_linear.argtypes = [vp, expert, vp, vp, vp, vp, vp, vp, vp]
    L.moe_expert_linear.restype = i32
    L.moe_expert_backward_workspace_bytes.argtypes = [vp, expert]
    L.moe_expert_backward_workspace_bytes.restype = sz
    L.moe_expert_linear_backward.argtypes = [vp, expert, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
    L.moe_expert_linear_backward.restype = i32
    norm = ctypes.POINTER(NormConfig)
    L.moe_norm.argtypes = [vp, norm, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_norm.restype = i32
    L.moe_norm_backward_workspace_bytes.argtypes = [vp, norm]
    L.moe_norm_backward_workspace_bytes.restype = sz
    L.moe_norm_backward.argtypes = [vp, norm, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_norm_backward.restype = i32
    w4 = ctypes.POINTER(Weights4Config)
    L.moe_weights4_bytes.argtypes = [w4]
    L.moe_weights4_bytes.restype = sz
    L.moe_weights4_pack.argtypes = [w4, vp, vp, vp, vp]
    L.moe_weights4_pack.restype = i32
    L.moe_weights4_quantize.argtypes = [w4, vp, vp, vp]
    L.moe_weights4_quantize.restype = i32
    L.moe_weights4_unpack.argtypes = [w4, vp, vp, i32, vp]
    L.moe_weights4_unpack.restype = i32
    L.moe_expert_linear4.argtypes = [vp, expert, w4, vp, vp, vp, vp, vp, vp]
    L.moe_expert_linear4.restype = i32
    L.moe_status_str.argtypes = [i32]
    L.moe_status_str.restype = ctypes.c_char_p
    _lib = L
    return L


def kernel_name(kernel: int) -> str:
    return lib().moe_kernel_name(kernel).decode()


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def check(status: int, what: str) -> None:
    if status != OK:
        raise MoeError(status, what)
