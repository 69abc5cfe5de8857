// Host side of the C ABI declared in include/moe_layer.h: argument checks and
// the launch sequence of each call.  Checks come before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "layer_internal.h"
#include "moe_plan.h"

namespace moe {
namespace {

bool is_dtype(int32_t v) { return v == MOE_OUT_BF16 || v == MOE_OUT_F32; }

bool good(const void* p, size_t a) { return p != nullptr && aligned(p, a); }

// Experts of the m smallest of the plan's nodes together.
int64_t fewest_experts(const Dims& d, int32_t m) {
  // The ranks with one expert more come first, so the last nodes are smallest.
  const int64_t r0 = (int64_t)(d.N - m) * d.G;
  return (int64_t)d.E - (r0 * d.ebase + std::min<int64_t>(r0, d.erem));
}

moe_status check_router(const moe_plan* plan, const moe_router_config* c, int32_t dtype) {
  if (!plan || !c || !is_dtype(dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARGUMENT;
  if (c->key != MOE_KEY_LOGIT && c->key != MOE_KEY_SCORE) return MOE_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(c->scale)) return MOE_ERR_INVALID_ARGUMENT;
  const Dims& d = plan->d;
  if (c->nodes_per_token < 0 || c->nodes_per_token > d.N) return MOE_ERR_INVALID_ARGUMENT;
  if (c->nodes_per_token > 0) {
    if (d.N > kRouterMaxNodes) return MOE_ERR_UNSUPPORTED;
    if (fewest_experts(d, c->nodes_per_token) < d.k) return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

constexpr int32_t kMaxFeatures = 1 << 20;
constexpr int64_t kMaxWeight = (int64_t)1 << 30;  // elements of one expert's weight

moe_status expert_dims(const moe_plan* plan, const moe_expert_config* c, ExpertDims* out) {
  if (!plan || !c) return MOE_ERR_INVALID_ARGUMENT;
  if (c->in_features <= 0 || c->in_features % 8 || c->out_features <= 0 || c->out_features % 8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_GEGLU) return MOE_ERR_INVALID_ARGUMENT;
  const Dims& d = plan->d;
  const int64_t Z = (int64_t)c->out_features * (gated(c->activation) ? 2 : 1);
  if (c->in_features > kMaxFeatures || Z > kMaxFeatures || Z * c->in_features >= kMaxWeight)
    return MOE_ERR_UNSUPPORTED;
  *out = ExpertDims{d.T * d.k, d.E,           c->in_features, c->out_features, (int32_t)Z,
                    d.T,       c->activation, d.nbands,       d.band};
  return MOE_OK;
}

// Workspace: grad_z in bf16 (with an activation), then the bias sums.
size_t gz_bytes(const ExpertDims& x) {
  if (x.act == MOE_ACT_NONE) return 0;
  return ((size_t)x.rows * x.Z * 2 + 255) / 256 * 256;
}

size_t partial_bytes(const ExpertDims& x) {
  return ((size_t)bias_slots(x) * x.Z * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_router(moe_plan* plan, const moe_router_config* cfg, const void* logits,
                      int32_t logits_dtype, const float* bias, int32_t* topk_idx, float* topk_w,
                      void* stream) {
  const moe_status st = moe::check_router(plan, cfg, logits_dtype);
  if (st != MOE_OK) return st;
  const moe::TimerScope timing(plan);
  if (plan->d.T == 0) return MOE_OK;
  const bool f32 = logits_dtype == MOE_OUT_F32;
  if (!moe::good(logits, f32 ? 4 : 2) || !moe::aligned(bias, 4) || !moe::good(topk_idx, 4) ||
      !moe::good(topk_w, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_router(plan->d, *cfg, logits, f32, bias, topk_idx, topk_w,
                                          static_cast<hipStream_t>(stream)));
}

moe_status moe_router_backward(moe_plan* plan, const moe_router_config* cfg, const void* logits,
                               int32_t logits_dtype, const int32_t* topk_idx, const float* grad_w,
                               void* grad_logits, void* stream) {
  const moe_status st = moe::check_router(plan, cfg, logits_dtype);
  if (st != MOE_OK) return st;
  const moe::TimerScope timing(plan);
  if (plan->d.T == 0) return MOE_OK;
  const bool f32 = logits_dtype == MOE_OUT_F32;
  if (!moe::good(logits, f32 ? 4 : 2) || !moe::good(topk_idx, 4) || !moe::good(grad_w, 4) ||
      !moe::good(grad_logits, f32 ? 4 : 2))
    return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_router_grad(plan->d, *cfg, logits, f32, topk_idx, grad_w,
                                               grad_logits, static_cast<hipStream_t>(stream)));
}

moe_status moe_dispatch_backward(moe_plan* plan, const uint16_t* grad_recv, void* grad_x,
                                 int32_t out_dtype, void* stream) {
  if (!plan) return MOE_ERR_INVALID_ARGUMENT;
  const moe::TimerScope timing(plan);
  if (!plan->routed) return MOE_ERR_PLAN_NOT_ROUTED;
  if (!moe::is_dtype(out_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (plan->d.T == 0) return MOE_OK;
  if (!moe::good(grad_recv, 16) || !moe::good(grad_x, 16)) return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe_status st = moe::ensure_assigned(plan, s);
  if (st != MOE_OK) return st;
  return moe::from_hip(moe::launch_dispatch_grad(plan->d, grad_recv, grad_x,
                                                 out_dtype == MOE_OUT_F32, plan->work, s));
}

moe_status moe_combine_backward(moe_plan* plan, const void* grad_out, int32_t grad_dtype,
                                const uint16_t* y, const float* topk_w, uint16_t* grad_y,
                                float* grad_w, void* stream) {
  if (!plan) return MOE_ERR_INVALID_ARGUMENT;
  const moe::TimerScope timing(plan);
  if (!plan->routed) return MOE_ERR_PLAN_NOT_ROUTED;
  if (!moe::is_dtype(grad_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (plan->d.T == 0) return MOE_OK;
  if (!moe::good(grad_out, 16) || !moe::good(y, 16) || !moe::good(topk_w, 4) ||
      !moe::good(grad_y, 16) || !moe::good(grad_w, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe_status st = moe::ensure_assigned(plan, s);
  if (st != MOE_OK) return st;
  return moe::from_hip(moe::launch_combine_grad(plan->d, grad_out, grad_dtype == MOE_OUT_F32, y,
                                                topk_w, grad_y, grad_w, plan->work, s));
}

moe_status moe_expert_linear(moe_plan* plan, const moe_expert_config* cfg, const uint16_t* x,
                             const uint16_t* w, const float* bias, const uint16_t* residual,
                             uint16_t* y, uint16_t* pre, void* stream) {
  moe::ExpertDims dims;
  const moe_status ok = moe::expert_dims(plan, cfg, &dims);
  if (ok != MOE_OK) return ok;
  const moe::TimerScope timing(plan);
  if (!plan->routed) return MOE_ERR_PLAN_NOT_ROUTED;
  if (plan->d.T == 0) return MOE_OK;
  if (!moe::good(x, 16) || !moe::good(w, 16) || !moe::aligned(bias, 16) ||
      !moe::aligned(residual, 16) || !moe::good(y, 16) || !moe::aligned(pre, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe_status st = moe::ensure_scanned(plan, s);
  if (st != MOE_OK) return st;
  return moe::from_hip(moe::launch_expert_rows(dims, plan->work.expert_off, x, w, bias, residual, y,
                                               pre, s));
}

size_t moe_expert_backward_workspace_bytes(const moe_plan* plan, const moe_expert_config* cfg) {
  moe::ExpertDims dims;
  if (moe::expert_dims(plan, cfg, &dims) != MOE_OK) return 0;
  return moe::gz_bytes(dims) + moe::partial_bytes(dims);
}

moe_status moe_expert_linear_backward(moe_plan* plan, const moe_expert_config* cfg,
                                      const uint16_t* grad_y, const uint16_t* x, const uint16_t* w,
                                      const uint16_t* pre, uint16_t* grad_x, void* grad_w,
                                      int32_t w_dtype, float* grad_bias, void* workspace,
                                      void* stream) {
  moe::ExpertDims dims;
  const moe_status ok = moe::expert_dims(plan, cfg, &dims);
  if (ok != MOE_OK) return ok;
  const moe::TimerScope timing(plan);
  if (!plan->routed) return MOE_ERR_PLAN_NOT_ROUTED;
  if (!moe::is_dtype(w_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  const bool act = dims.act != MOE_ACT_NONE, empty = plan->d.T == 0;
  if (!moe::aligned(grad_x, 16) || !moe::aligned(grad_w, 16) || !moe::aligned(grad_bias, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!moe::good(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
  if (!empty && (!moe::good(grad_y, 16) || (act && !moe::good(pre, 16)) ||
                 (grad_x && !moe::good(w, 16)) || (grad_w && !moe::good(x, 16))))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe_status st = moe::ensure_scanned(plan, s);
  if (st != MOE_OK) return st;
  const int32_t* off = plan->work.expert_off;
  uint16_t* gz = static_cast<uint16_t*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + moe::gz_bytes(dims));
  const bool products = grad_x || grad_w;
  hipError_t e = hipSuccess;
  if (!empty && ((act && products) || grad_bias))
    e = moe::launch_expert_act_grad(dims, off, grad_y, pre, act && products ? gz : nullptr,
                                    grad_bias ? partial : nullptr, s);
  const uint16_t* g = act ? gz : grad_y;
  const bool f32 = w_dtype == MOE_OUT_F32;
  if (e == hipSuccess && grad_w && grad_x && !empty)
    return moe::from_hip(moe::launch_expert_grads(dims, off, g, w, grad_x, x, grad_w, f32, partial,
                                                  grad_bias, s));
  if (e == hipSuccess && grad_bias) e = moe::launch_expert_bias_sum(dims, off, partial, grad_bias, s);
  if (e == hipSuccess && grad_w)
    e = moe::launch_expert_wgrad(dims, off, g, x, grad_w, f32, s);
  if (e == hipSuccess && grad_x && !empty)
    e = moe::launch_expert_rows_grad(dims, off, g, w, grad_x, s);
  return moe::from_hip(e);
}

}  // extern "C"
