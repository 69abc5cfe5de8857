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

constexpr int32_t kMaxFeatures = 1 << 20;
constexpr int64_t kMaxWeight = (int64_t)1 << 30;  // elements of one expert's weight

moe_status weights4(const moe_weights4_config* c, Weights4* out) {
  if (!c) return MOE_ERR_INVALID_ARGUMENT;
  if (c->experts <= 0 || c->rows <= 0 || c->rows % 8 || c->in_features <= 0 || c->in_features % 8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (c->format != MOE_W4_INT4 && c->format != MOE_W4_E2M1) return MOE_ERR_INVALID_ARGUMENT;
  const bool e2m1 = c->format == MOE_W4_E2M1;
  if (c->group != 32 && (e2m1 || (c->group != 64 && c->group != 128)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (c->experts > MOE_MAX_EXPERTS || c->rows > kMaxFeatures || c->in_features > kMaxFeatures ||
      (int64_t)c->rows * c->in_features >= kMaxWeight)
    return MOE_ERR_UNSUPPORTED;
  *out = Weights4{c->experts, c->rows,  c->in_features, e2m1,
                  c->group,   (c->in_features + 127) / 128, (c->rows + 15) / 16};
  return MOE_OK;
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

size_t moe_weights4_bytes(const moe_weights4_config* cfg) {
  moe::Weights4 w;
  return moe::weights4(cfg, &w) == MOE_OK ? (size_t)(w.codes_bytes() + w.scales_bytes()) : 0;
}

moe_status moe_weights4_pack(const moe_weights4_config* cfg, const uint8_t* codes,
                             const void* scales, void* packed, void* stream) {
  moe::Weights4 w;
  const moe_status ok = moe::weights4(cfg, &w);
  if (ok != MOE_OK) return ok;
  if (!moe::good(codes, 16) || !moe::good(scales, w.e2m1 ? 1 : 2) || !moe::good(packed, 256))
    return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_pack4(w, codes, scales, packed, static_cast<hipStream_t>(stream)));
}

moe_status moe_weights4_quantize(const moe_weights4_config* cfg, const uint16_t* from, void* packed,
                                 void* stream) {
  moe::Weights4 w;
  const moe_status ok = moe::weights4(cfg, &w);
  if (ok != MOE_OK) return ok;
  if (!moe::good(from, 16) || !moe::good(packed, 256)) return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_quantize4(w, from, packed, static_cast<hipStream_t>(stream)));
}

moe_status moe_weights4_unpack(const moe_weights4_config* cfg, const void* packed, void* to,
                               int32_t w_dtype, void* stream) {
  moe::Weights4 w;
  const moe_status ok = moe::weights4(cfg, &w);
  if (ok != MOE_OK) return ok;
  if (!moe::is_dtype(w_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (!moe::good(packed, 256) || !moe::good(to, 16)) return MOE_ERR_INVALID_ARGUMENT;
  return moe::from_hip(moe::launch_unpack4(w, packed, to, w_dtype == MOE_OUT_F32,
                                           static_cast<hipStream_t>(stream)));
}

moe_status moe_expert_linear4(moe_plan* plan, const moe_expert_config* cfg,
                              const moe_weights4_config* w4, const uint16_t* x, const void* packed,
                              const float* bias, const uint16_t* residual, uint16_t* y,
                              void* stream) {
  if (!plan || !cfg) return MOE_ERR_INVALID_ARGUMENT;
  moe::Weights4 w;
  const moe_status ok = moe::weights4(w4, &w);
  if (ok != MOE_OK) return ok;
  if (cfg->activation < MOE_ACT_NONE || cfg->activation > MOE_ACT_GEGLU || cfg->out_features <= 0 ||
      cfg->out_features % 8)
    return MOE_ERR_INVALID_ARGUMENT;
  const moe::Dims& d = plan->d;
  const int64_t Z = (int64_t)cfg->out_features * (moe::gated(cfg->activation) ? 2 : 1);
  if (w.E != d.E || w.Z != Z || w.K != cfg->in_features) return MOE_ERR_INVALID_ARGUMENT;
  const moe::TimerScope timing(plan);
  if (!plan->routed) return MOE_ERR_PLAN_NOT_ROUTED;
  if (d.T == 0) return MOE_OK;
  if (!moe::good(x, 16) || !moe::good(packed, 256) || !moe::aligned(bias, 16) ||
      !moe::aligned(residual, 16) || !moe::good(y, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  const moe::ExpertDims dims{d.T * d.k, d.E,            w.K,      cfg->out_features, (int32_t)Z,
                             d.T,       cfg->activation, d.nbands, d.band};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe_status st = moe::ensure_scanned(plan, s);
  if (st != MOE_OK) return st;
  return moe::from_hip(moe::launch_expert_rows4(dims, w, plan->work.expert_off, x, packed, bias,
                                                residual, y, s));
}

}  // extern "C"
