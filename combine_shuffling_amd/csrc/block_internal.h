// Internal declarations of the operators of moe_block.h (moe_block_api.cpp and
// norm.hip, weights4.hip, expert4.h).  Not part of the public ABI.
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

// ---- 4-bit weights
//
// Packed layout.  A weight row is cut into blocks of 128 along K (the last is
// padded with weights of 0); a block is 64 bytes, a row's blocks and an
// expert's rows follow each other.  The 32-bit word g * 4 + s of a block holds the
// eight weights 32 s + 8 g + 0..7: 16 bytes are what one lane of lane group g
// multiplies in the block's four matrix instructions s of 32 weights.  In a word E2M1
// weight i is nibble i, as the conversion instruction takes them; INT4 weight 2p is
// nibble p and weight 2p + 1 nibble p + 4, so that one shift and one mask leave
// a pair of them in the halves of a register.
// Scales follow at a multiple of 256 bytes: INT4 [E, groups, Z] bf16 (a
// lane's results are consecutive rows of w), E2M1 [E, Z, groups] bytes (a
// block's four scales are one word); groups are those of the padded row.
struct Weights4 {
  int32_t E, Z, K;
  int32_t e2m1;      // format
  int32_t group;
  int32_t blocks;    // of 128 along K
  __host__ __device__ int groups() const { return blocks * (128 / group); }
  __host__ __device__ int given_groups() const { return (K + group - 1) / group; }
  __host__ __device__ int64_t row_bytes() const { return (int64_t)blocks * 64; }
  __host__ __device__ int64_t codes_bytes() const { return (E * row_bytes() * Z + 255) / 256 * 256; }
  __host__ __device__ int64_t scales_bytes() const {
    return ((int64_t)E * Z * groups() * (e2m1 ? 1 : 2) + 255) / 256 * 256;
  }
};

hipError_t launch_pack4(const Weights4& w, const uint8_t* codes, const void* scales, void* packed,
                        hipStream_t s);
hipError_t launch_quantize4(const Weights4& w, const uint16_t* from, void* packed, hipStream_t s);
hipError_t launch_unpack4(const Weights4& w, const void* packed, void* to, bool f32, hipStream_t s);

// expert4.h (in expert.hip)
hipError_t launch_expert_rows4(const ExpertDims& x, const Weights4& w4, const int32_t* off,
                               const uint16_t* a, const void* packed, const float* bias,
                               const uint16_t* residual, uint16_t* y, hipStream_t s);

}  // namespace moe
