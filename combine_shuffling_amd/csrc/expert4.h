// The experts' products with 4-bit weights (included at the end of expert.hip, whose tables,
// activations and tile product they use): z = x w[e]^T for every expert e with receive rows
// [off[e], off[e + 1]), w = scale * code.  The layout of the packed weights is described in
// block_internal.h.
#pragma once

namespace moe {
namespace {

// ---- codes to bf16

// Eight E2M1 codes times 2^(scale - 127), exact (bf16 has the range of the scales; a value past it
// is infinite, a scale of 255 gives NaN): the conversion instruction reads the scale's exponent.
__device__ __forceinline__ bf16x8 decode_e2m1(uint32_t codes, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return __builtin_bit_cast(bf16x8, r);
}

__device__ __forceinline__ float e2m1_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight INT4 codes c (0..15) as the bf16 numbers 128 + c: the code is the low bits of the mantissa
// under the exponent of 128.
constexpr float kInt4Offset = 136.0f;  // 128 + c stands for c - 8
__device__ __forceinline__ bf16x8 decode_int4(uint32_t codes) {
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = ((codes >> (4 * p)) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, r);
}

// ---- few rows an expert

// Which expert a block of the few-rows kernels works on: `which`, or, where a batch (or band) has
// fewer rows than experts, that of row `which` if it is the expert's first; else -1.
__device__ __forceinline__ int few_rows_expert(const ExpertDims& x, const int32_t* off, int which) {
  if (x.rows >= x.E) return which;
  const int lane = threadIdx.x % kWave;
  const int row = off[0] + which;
  const int step = (x.E + kWave - 1) / kWave;
  const int e1 = lane * step;
  int e = (__popcll(__ballot(e1 < x.E && off[min(e1, x.E)] <= row)) - 1) * step;
  if (step > 1) {
    const int e2 = e + lane;
    e += __popcll(__ballot(lane < step && e2 < x.E && off[min(e2, x.E)] <= row)) - 1;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  return off[e] == row ? e : -1;
}

// One block computes 16 columns of y with a gated activation (16 of the gate and 16 of the up
// projection), else 32, for one expert: two strips of 16 weight rows.  Its waves split the
// contraction in blocks of 128, read codes and rows straight into matrix-instruction registers and
// add their parts through LDS in a fixed order.  MT * 16 rows a pass; an expert with more takes
// further passes.
//
// E2M1 weights are exact in bf16, scale and all.  INT4: the sums of a group's products with 128 + c
// and with -136 are added up in float32, which leaves the sum with c - 8, and the scale multiplies
// that sum: no weight is rounded.
template <int G, bool E2M1, int MT, bool GATED>
__global__ __launch_bounds__(kFewWaves * kWave) void expert4_few_rows_kernel(
    ExpertDims x, Weights4 w4, const int32_t* __restrict__ off, const char* __restrict__ a,
    const char* __restrict__ codes, const char* __restrict__ scales, const float* __restrict__ bias,
    const uint16_t* __restrict__ residual, uint16_t* __restrict__ y, int strips, int64_t base) {
  constexpr int kAhead = 4 / MT;          // blocks of 128 loaded together
  constexpr int kGroups = 128 / G;        // scales a block
  constexpr int kCols = GATED ? 16 : 32;  // columns of y
  __shared__ float part[kFewWaves][MT * 2][256];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t block = base + blockIdx.x;
  const int e = few_rows_expert(x, off, (int)(block / strips));
  if (e < 0) return;
  const int col0 = (int)(block % strips) * kCols;
  const int o0 = off[e], rows = off[e + 1] - o0;
  const uint32_t ld = (uint32_t)x.K * 2, ldw = (uint32_t)w4.blocks * 64;
  const int first = wave * w4.blocks / kFewWaves, last = (wave + 1) * w4.blocks / kFewWaves;
  const int i = lane & 15, g = lane >> 4;
  const uint32_t second = GATED ? x.N : 16;  // weight rows from the first strip to the second
  const __amdgpu_buffer_rsrc_t rw =
      uniform_buffer(codes + (int64_t)e * x.Z * ldw, (uint32_t)x.Z * ldw);
  const int64_t scale_bytes = (int64_t)w4.groups() * x.Z * (E2M1 ? 1 : 2);
  const __amdgpu_buffer_rsrc_t rs = uniform_buffer(scales + e * scale_bytes, (uint32_t)scale_bytes);
  // (Weight rows past the last give results that are not stored, or are past the descriptor's end.)
  const uint32_t vw = (uint32_t)(col0 + i) * ldw + g * 16;
  const uint32_t vs = E2M1 ? (uint32_t)(col0 + i) * w4.blocks * 4 : (uint32_t)(col0 + g * 4) * 2;
  bf16x8 offset;
#pragma unroll
  for (int q = 0; q < 8; ++q) offset[q] = (__bf16)-kInt4Offset;
  for (int r0 = 0; r0 < rows; r0 += MT * 16) {
    const __amdgpu_buffer_rsrc_t rx = uniform_buffer(
        a + (int64_t)(o0 + r0) * ld, (uint32_t)min(rows - r0, MT * 16) * ld);  // rows past the end: zeros
    f32x4 acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc[m][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = first; b0 < last; b0 += kAhead) {
      u32x4 cw[kAhead][2];
      u32x2 si[kAhead][2][kGroups];  // INT4: the scales of the lane's four result columns
      uint32_t se[kAhead][2];        // E2M1: those of the lane's weight row
      bf16x8 fx[kAhead][4][MT];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool in = b0 + u < last;
        const uint32_t b = (uint32_t)(b0 + u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cw[u][h] = __builtin_amdgcn_raw_buffer_load_b128(
              rw, in ? vw + h * second * ldw + b * 64 : kPast, 0, 0);
          if constexpr (E2M1)
            se[u][h] = __builtin_amdgcn_raw_buffer_load_b32(
                rs, in ? vs + (h * second * w4.blocks + b) * 4 : kPast, 0, 0);
          else
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
              si[u][h][q] = __builtin_amdgcn_raw_buffer_load_b64(
                  rs, in ? vs + ((b * kGroups + q) * x.Z + h * second) * 2 : kPast, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = (b0 + u) * 128 + s * 32 + g * 8;
          const bool in = b0 + u < last && k < x.K;  // chunks past a row's end read zeros
#pragma unroll
          for (int m = 0; m < MT; ++m)
            fx[u][s][m] = __builtin_bit_cast(
                bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                            rx, in ? (uint32_t)(m * 16 + i) * ld + k * 2 : kPast, 0, 0));
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if constexpr (E2M1) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bf16x8 f = decode_e2m1(cw[u][h][s], e2m1_scale((se[u][h] >> (8 * s)) & 0xffu));
#pragma unroll
              for (int m = 0; m < MT; ++m)
                acc[m][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, fx[u][s][m], acc[m][h], 0, 0, 0);
            }
        } else {
#pragma unroll
          for (int q = 0; q < kGroups; ++q) {
            f32x4 less[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              less[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int s = q * G / 32; s < (q + 1) * G / 32; ++s)
                less[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(offset, fx[u][s][m], less[m], 0, 0, 0);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f32x4 sum[MT];
#pragma unroll
              for (int m = 0; m < MT; ++m) sum[m] = less[m];
#pragma unroll
              for (int s = q * G / 32; s < (q + 1) * G / 32; ++s) {
                const bf16x8 f = decode_int4(cw[u][h][s]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, fx[u][s][m], sum[m], 0, 0, 0);
              }
              const u32x2 v = si[u][h][q];
              const float sc[4] = {__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u),
                                   __uint_as_float(v[1] << 16), __uint_as_float(v[1] & 0xffff0000u)};
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  acc[m][h][c] = __builtin_fmaf(sc[c], sum[m][c], acc[m][h][c]);
            }
          }
        }
      }
    }
    // acc[m][h][q]: column g * 4 + q of strip h, row m * 16 + i.
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4*>(&part[wave][m * 2 + h][i * 16 + g * 4]) = acc[m][h];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 16 * kCols; t += kFewWaves * kWave) {
      const int r = r0 + t / kCols, c = t % kCols, col = col0 + c;
      if (r >= rows || col >= x.N) continue;
      const int m = t / kCols / 16, at = t / kCols % 16 * 16 + c % 16;
      float z[2];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        z[h] = 0.0f;
#pragma unroll
        for (int q = 0; q < kFewWaves; ++q) z[h] += part[q][m * 2 + (GATED ? h : c / 16)][at];
        if (bias != nullptr) z[h] += bias[(int64_t)e * x.Z + h * x.N + col];
      }
      const int64_t row = o0 + r;
      float out[8] = {z[0]};
      act_values(x.act, out);
      if constexpr (GATED) out[0] *= z[1];
      if (residual != nullptr)
        out[0] += __uint_as_float((uint32_t)residual[row * x.N + col] << 16);
      y[row * x.N + col] = (uint16_t)bf16_pair(out[0], 0.0f);
    }
    __syncthreads();
  }
}

hipError_t expert_rows4(const ExpertDims& x, const Weights4& w4, const int32_t* off,
                        const uint16_t* a, const void* packed, const float* bias,
                        const uint16_t* residual, uint16_t* y, hipStream_t s) {
  const char* codes = static_cast<const char*>(packed);
  const char* scales = codes + w4.codes_bytes();
  auto few = [&](auto kernel) {
    const int strips = ceil_div(x.N, gated(x.act) ? 16 : 32);
    return in_ranges((int64_t)std::min(x.E, x.rows) * strips, [&](dim3 blocks, int64_t b) {
      return launch(MOE_KERNEL_EXPERT4_FEW_ROWS, kernel, blocks, dim3(kFewWaves * kWave), 0, s, x, w4,
                    off, reinterpret_cast<const char*>(a), codes, scales, bias, residual, y, strips, b);
    });
  };
  auto by_rows = [&](auto group, auto e2m1) {
    constexpr int G = decltype(group)::value;
    constexpr bool E2M1 = decltype(e2m1)::value;
    if (x.T <= 16 || (int64_t)x.rows <= (int64_t)x.E * (kFewRows / 2))
      return gated(x.act) ? few(expert4_few_rows_kernel<G, E2M1, 1, true>)
                          : few(expert4_few_rows_kernel<G, E2M1, 1, false>);
    return gated(x.act) ? few(expert4_few_rows_kernel<G, E2M1, 2, true>)
                        : few(expert4_few_rows_kernel<G, E2M1, 2, false>);
  };
  if (w4.e2m1) return by_rows(std::integral_constant<int, 32>(), std::true_type());
  if (w4.group == 32) return by_rows(std::integral_constant<int, 32>(), std::false_type());
  if (w4.group == 64) return by_rows(std::integral_constant<int, 64>(), std::false_type());
  return by_rows(std::integral_constant<int, 128>(), std::false_type());
}

}  // namespace

hipError_t launch_expert_rows4(const ExpertDims& x, const Weights4& w4, const int32_t* off,
                               const uint16_t* a, const void* packed, const float* bias,
                               const uint16_t* residual, uint16_t* y, hipStream_t s) {
  return by_band(x, off, [&](const ExpertDims& xb, const int32_t* ob, int) {
    return expert_rows4(xb, w4, ob, a, packed, bias, residual, y, s);
  });
}

}  // namespace moe
