/*
 * moe_block.h -- what stands around the Mixture-of-Experts layer of
 * moe_layer.h in a transformer block on one MI355X (gfx950): the norm of the
 * residual stream in front of the router and the dispatch, with its gradient,
 * and the experts' products with weights of 4 bits for serving.  Same library,
 * plans, statuses and conventions.
 *
 *   moe_norm               residual addition, then layer norm or RMS norm
 *   moe_norm_backward      its gradient
 *   moe_weights4_pack      4-bit codes and scales -> packed weights
 *   moe_weights4_quantize  bf16 weights -> packed weights
 *   moe_weights4_unpack    the values that packed weights stand for
 *   moe_expert_linear4     moe_expert_linear with packed weights
 *
 * A decoding step calls moe_norm, moe_router on the gate's logits,
 * moe_route_plan, moe_dispatch, moe_expert_linear4 (once for each product) and
 * moe_combine, whose output is the residual of the next block's moe_norm.
 * Arguments, streams and errors as in moe_layer.h: contiguous device buffers
 * of the caller, 16-byte aligned unless said otherwise, distinct from those
 * the call writes; asynchronous, nothing is allocated, no atomics on floating
 * values.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- norm ------------------------------------------------------------------ */

typedef enum moe_norm_kind {
  MOE_NORM_LAYER = 0, /* the mean is taken off      */
  MOE_NORM_RMS = 1    /* mean = 0 in the formulas   */
} moe_norm_kind;

typedef struct moe_norm_config {
  int32_t kind;    /* moe_norm_kind                                       */
  float eps;       /* >= 0, finite; added to the variance                 */
  int32_t x_dtype; /* moe_out_dtype of x, residual, total and grad_x      */
  int32_t y_dtype; /* moe_out_dtype of y and grad_y                       */
} moe_norm_config;

/* Norm of the plan's T rows of H columns:
 *   total = x + residual             float32 sum, rounded to x_dtype
 *   mean  = sum(total) / H           (RMS: 0)
 *   rstd  = 1 / sqrt(sum((total - mean)^2) / H + eps)
 *   y     = (total - mean) * rstd * gamma + beta
 * in float32 from the rounded total, y rounded to y_dtype (nearest even).
 * x, residual, total: [T, H]; residual NULL: total = x, and total has to be
 * NULL.  total may be NULL with a residual too (not wanted).  gamma, beta: [H]
 * float32, NULL for ones and zeros.  y: [T, H].  stats: [T, 2] float32, mean
 * and rstd, as the gradient takes them, 8-byte aligned, or NULL.
 * A row whose sum of squares passes float32's range has rstd 0, and one whose
 * sum does (layer norm) NaN for y.  The plan need not be routed; its experts
 * take no part.  Limit: H <= 16384.
 * Errors: INVALID_ARGUMENT (null or misaligned pointers, unknown kind or
 * dtype, eps negative or not finite, a total without a residual), UNSUPPORTED
 * (H beyond the limit), HIP. */
moe_status moe_norm(moe_plan* plan, const moe_norm_config* cfg, const void* x, const void* residual,
                    const float* gamma, const float* beta, void* y, void* total, float* stats,
                    void* stream);

/* Device workspace of moe_norm_backward (bytes, a multiple of 256; it may be
 * 0): the partial sums of the weights' gradients.  Its contents need no
 * initialisation.  0 for a cfg that the call refuses. */
size_t moe_norm_backward_workspace_bytes(const moe_plan* plan, const moe_norm_config* cfg);

/* Gradient of moe_norm.  With h = (total - mean) * rstd and g = grad_y * gamma:
 *   grad_x = rstd * (g - mean_H(g) - h * mean_H(g * h)) + grad_total
 *            (RMS: without mean_H(g)), rounded to x_dtype
 *   grad_gamma = sum over the rows of grad_y * h        float32 [H]
 *   grad_beta  = sum over the rows of grad_y            float32 [H]
 * Each may be NULL (not wanted); without rows the sums are zeros.  grad_x is
 * the gradient of x and of the residual.  total: what was normed (x without a
 * residual); stats: as moe_norm stored them; grad_total: [T, H] of x_dtype,
 * the gradient that reaches total by other ways, or NULL; workspace: 256-byte
 * aligned, may be NULL where its size is 0.  cfg->eps is only checked.
 * Errors as moe_norm. */
moe_status moe_norm_backward(moe_plan* plan, const moe_norm_config* cfg, const void* grad_y,
                             const void* total, const float* stats, const float* gamma,
                             const void* grad_total, void* grad_x, float* grad_gamma,
                             float* grad_beta, void* workspace, void* stream);

/* ---- the experts' products with 4-bit weights -------------------------------- */

typedef enum moe_weights4_format {
  MOE_W4_INT4 = 0, /* w = scale * (code - 8), scale bf16, a scale per group of 32, 64 or 128        */
  MOE_W4_E2M1 = 1  /* w = 2^(scale - 127) * OCP E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
                      negatives), scale E8M0 (255: NaN), a scale per group of 32              */
} moe_weights4_format;

typedef struct moe_weights4_config {
  int32_t experts;     /* E > 0                                                      */
  int32_t rows;        /* Z > 0, multiple of 8: weight rows an expert                */
  int32_t in_features; /* K > 0, multiple of 8                                       */
  int32_t format;      /* moe_weights4_format                                        */
  int32_t group;       /* weights of a row that share a scale; a row's last group may have fewer */
} moe_weights4_config;

/* Packed weights: codes in the order in which the matrix cores take them, and
 * scales, in one device buffer of moe_weights4_bytes (a multiple of 256; 0 for
 * a cfg that the calls refuse), 256-byte aligned.  The layout is the library's
 * own.
 * Limits of these calls: E <= MOE_MAX_EXPERTS, Z * K < 2^30, K and Z <= 2^20.
 * Errors of all of them: INVALID_ARGUMENT, UNSUPPORTED (sizes beyond the
 * limits), HIP. */
size_t moe_weights4_bytes(const moe_weights4_config* cfg);

/* Packs codes as a checkpoint holds them.  codes: [E, Z, K / 2] uint8, weight
 * 2j in the lower nibble of byte j; scales: [E, Z, ceil(K / group)] bf16
 * (INT4) or uint8 (E2M1). */
moe_status moe_weights4_pack(const moe_weights4_config* cfg, const uint8_t* codes,
                             const void* scales, void* packed, void* stream);

/* Quantizes bf16 weights w [E, Z, K].  INT4: scale = max |w| / 7 over the group,
 * rounded to bf16; code - 8 = w / scale rounded to nearest even, within -8 and
 * 7.  E2M1: scale = the smallest power of two with max |w| <= 6 * scale (within
 * E8M0's range; 1 for a group of zeros); code = w / scale rounded to nearest
 * (ties to the even code).  A group that holds an infinity or a NaN gets the
 * scale NaN. */
moe_status moe_weights4_quantize(const moe_weights4_config* cfg, const uint16_t* w, void* packed,
                                 void* stream);

/* The values that packed weights stand for: w [E, Z, K] of w_dtype
 * (moe_out_dtype; scale * code is rounded once, to it). */
moe_status moe_weights4_unpack(const moe_weights4_config* cfg, const void* packed, void* w,
                               int32_t w_dtype, void* stream);

/* Expert product with packed weights, for serving (it has no gradient): for
 * every receive row r of expert e,
 *   z[r] = x[r] . w[e]^T + bias[e]        (float32 accumulation)
 *   y[r] = act(z[r]) + residual[r]        rounded to bf16 (nearest even)
 * No weight is rounded: E2M1 weights are bf16 numbers, subnormal ones too (and
 * infinite from 2^128 on), and of INT4 weights the codes are multiplied, and a
 * group's float32 sum by its scale.  (That sum is the difference of sums of
 * products with 16 + code and with 24: it rounds as sums of their magnitude do,
 * and x has to stay below 2^116.)  Arguments as moe_expert_linear; w4->experts,
 * rows and in_features are the plan's E and cfg's Z and K.  A row of x with an
 * infinity or a NaN gives a row that is not finite.  INT4 in groups of 32 is for
 * batches of few rows an expert: large ones take two to three times as long as
 * with groups of 64 or 128, and up to seven times where one expert has most rows.
 * Errors: PLAN_NOT_ROUTED, INVALID_ARGUMENT, UNSUPPORTED (sizes beyond the
 * limits), HIP. */
moe_status moe_expert_linear4(moe_plan* plan, const moe_expert_config* cfg,
                              const moe_weights4_config* w4, const uint16_t* x, const void* packed,
                              const float* bias, const uint16_t* residual, uint16_t* y,
                              void* stream);

/* Kernels of these calls, as moe_plan_timing_read names them (moe_kernel_name
 * takes their ids too). */
typedef enum moe_block_kernel {
  MOE_KERNEL_NORM = 64,
  MOE_KERNEL_NORM_GRAD,
  MOE_KERNEL_NORM_SUM,         /* partial sums of the weights' gradients added up  */
  MOE_KERNEL_EXPERT4_ROWS,     /* product with 4-bit weights                       */
  MOE_KERNEL_EXPERT4_FEW_ROWS, /* the same for batches of few rows an expert       */
  MOE_BLOCK_KERNEL_END
} moe_block_kernel;

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
