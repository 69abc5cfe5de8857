// Internal declarations of the operators of moe_block.h (moe_block_api.cpp and
// norm.hip).  Not part of the public ABI.
#pragma once

#include "layer_internal.h"
#include "moe_block.h"

namespace moe {

constexpr int kNormMaxColumns = 16384;

struct NormDims {
  int32_t T, H;
  int32_t rms;        // no mean
  float eps;
  bool x_f32, y_f32;  // types of the stream's rows and of y (or grad_y)
};

// Rows of partial sums that launch_norm_grad leaves (1: none, it writes the
// sums themselves).
int norm_partials(const NormDims& n);

hipError_t launch_norm(const NormDims& n, const void* x, const void* residual, const float* gamma,
                       const float* beta, void* y, void* total, float* stats, hipStream_t s);
// partial: [2, norm_partials, H] float32.
hipError_t launch_norm_grad(const NormDims& n, const void* gy, const void* total,
                            const float* stats, const float* gamma, const void* gtotal, void* gx,
                            float* ggamma, float* gbeta, float* partial, hipStream_t s);

}  // namespace moe
