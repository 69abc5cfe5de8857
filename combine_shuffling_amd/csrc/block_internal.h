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
// Packed layout.  An expert's weight rows are cut into tiles of 16 rows by 128 along K, which
// follow each other along K, then along the rows; rows and K are padded with weights of 0.  A
// tile is 1024 bytes: 16 for each lane of the wave that multiplies it, so that a load takes 1024
// consecutive bytes (lanes that each read 16 bytes of a row of their own cost the first-level
// cache a lookup each; a decoding step of 55 experts of 2048 x 2048 took 41 us that way, bound by
// them).  Lane 16 g + i has row i, and in word s of its four the weights 32 s + 8 g + 0..7, which
// are what it multiplies in the tile's matrix instruction s of 32 weights.  In a word E2M1 weight
// j is nibble j, as the conversion instruction takes them; INT4 weight 2p is nibble p and weight
// 2p + 1 nibble p + 4 of a word that is then rotated left by 3, so that one rotation by 4p and one mask
// leave a pair of them as the upper mantissa bits of the bf16 numbers in the halves of a register.
// Scales follow at a multiple of 256 bytes, tile by tile in the same order, so that a lane finds those
// of its row (E2M1, bytes: [16 rows][4 groups]), or of the four consecutive rows that its results are
// (INT4, bf16: [16 rows], [16 rows][2 groups], or two of these with groups of 32), side by side.
struct Weights4 {
  int32_t E, Z, K;
  int32_t e2m1;      // format
  int32_t group;
  int32_t blocks;    // of 128 along K
  int32_t tiles;     // of 16 rows
  __host__ __device__ int given_groups() const { return (K + group - 1) / group; }
  // Groups of a row whose scales are side by side.
  __host__ __device__ int beside() const { return e2m1 ? 4 : group == 128 ? 1 : 2; }
  // Bytes of one tile of 16 rows along all of K.
  __host__ __device__ uint32_t codes_stride() const { return (uint32_t)blocks * 1024; }
  __host__ __device__ uint32_t scales_stride() const {
    return (uint32_t)blocks * (e2m1 ? 64 : 128 / group * 32);
  }
  __host__ __device__ int64_t codes_bytes() const { return (int64_t)E * tiles * codes_stride(); }
  __host__ __device__ int64_t scales_bytes() const {
    return ((int64_t)E * tiles * scales_stride() + 255) / 256 * 256;
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
