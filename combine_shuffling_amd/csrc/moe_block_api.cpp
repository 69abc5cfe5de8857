// Host side of the C ABI declared in include/moe_block.h: argument checks and
// the launches of each call.  Checks come before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "block_internal.h"
#include "moe_plan.h"

namespace moe {
namespace {

bool is_dtype(int32_t v) { return v == MOE_OUT_BF16 || v == MOE_OUT_F32; }

bool good(const void* p, size_t a) { return p != nullptr && aligned(p, a); }

moe_status norm_dims(const moe_plan* plan, const moe_norm_config* c, NormDims* out) {
  if (!plan || !c) return MOE_ERR_INVALID_ARGUMENT;
  if (c->kind != MOE_NORM_LAYER && c->kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARGUMENT;
  if (!is_dtype(c->x_dtype) || !is_dtype(c->y_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(c->eps) || c->eps < 0.0f) return MOE_ERR_INVALID_ARGUMENT;
  if (plan->d.H > kNormMaxColumns) return MOE_ERR_UNSUPPORTED;
  *out = NormDims{plan->d.T, plan->d.H, c->kind == MOE_NORM_RMS, c->eps,
                  c->x_dtype == MOE_OUT_F32, c->y_dtype == MOE_OUT_F32};
  return MOE_OK;
}

size_t norm_workspace(const NormDims& n) {
  const int p = norm_partials(n);
  return p > 1 ? ((size_t)2 * p * n.H * sizeof(float) + 255) / 256 * 256 : 0;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_norm(moe_plan* plan, const moe_norm_config* cfg, const void* x, const void* residual,
                    const float* gamma, const float* beta, void* y, void* total, float* stats,
                    void* stream) {
  moe::NormDims n;
  const moe_status ok = moe::norm_dims(plan, cfg, &n);
  if (ok != MOE_OK) return ok;
  if (total && !residual) return MOE_ERR_INVALID_ARGUMENT;
  const moe::TimerScope timing(plan);
  if (n.T == 0) return MOE_OK;
  if (!moe::good(x, 16) || !moe::aligned(residual, 16) || !moe::aligned(gamma, 16) ||
      !moe::aligned(beta, 16) || !moe::good(y, 16) || !moe::aligned(total, 16) ||
      !moe::aligned(stats, 8))
    return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_norm(n, x, residual, gamma, beta, y, total, stats,
                                        static_cast<hipStream_t>(stream)));
}

size_t moe_norm_backward_workspace_bytes(const moe_plan* plan, const moe_norm_config* cfg) {
  moe::NormDims n;
  return moe::norm_dims(plan, cfg, &n) == MOE_OK ? moe::norm_workspace(n) : 0;
}

moe_status moe_norm_backward(moe_plan* plan, const moe_norm_config* cfg, const void* grad_y,
                             const void* total, const float* stats, const float* gamma,
                             const void* grad_total, void* grad_x, float* grad_gamma,
                             float* grad_beta, void* workspace, void* stream) {
  moe::NormDims n;
  const moe_status ok = moe::norm_dims(plan, cfg, &n);
  if (ok != MOE_OK) return ok;
  const moe::TimerScope timing(plan);
  const bool sums = grad_gamma || grad_beta;
  if (!moe::aligned(gamma, 16) || !moe::aligned(grad_total, 16) || !moe::aligned(grad_x, 16) ||
      !moe::aligned(grad_gamma, 16) || !moe::aligned(grad_beta, 16) ||
      !moe::aligned(workspace, 256))
    return MOE_ERR_INVALID_ARGUMENT;
  if (sums && !workspace && moe::norm_workspace(n) > 0) return MOE_ERR_INVALID_ARGUMENT;
  if (n.T > 0 && (!moe::good(grad_y, 16) || !moe::good(total, 16) || !moe::good(stats, 8)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!sums && (!grad_x || n.T == 0)) return MOE_OK;
  return moe::from_hip(moe::launch_norm_grad(n, grad_y, total, stats, gamma, grad_total, grad_x,
                                             grad_gamma, grad_beta, static_cast<float*>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
