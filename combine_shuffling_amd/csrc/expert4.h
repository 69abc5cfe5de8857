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
  uint32_t magic = 0x43004300u;
  asm("" : "+v"(magic));  // in a vector register: an instruction takes one constant of another kind
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = ((codes >> (4 * p)) & 0x000f000fu) | magic;
  return __builtin_bit_cast(bf16x8, r);
}

// The same codes times a scale, in bf16: the matrix instructions of a tile of many rows take the
// weights with their scales in them, since scaling sums of a group instead would take a second set of
// accumulators, for which there are no registers.  scale * (c - 8) is rounded to bf16 (nearest
// even), the one rounding of a weight; it is exact where the scale has five significant bits or fewer.
// The codes are first put under the exponent of 1024 in float16, from where one mixed multiply-add
// a code takes them: scale * (1024 + c) - 1032 * scale is exact in float32.
__device__ __forceinline__ bf16x8 decode_int4_scaled(uint32_t codes, float scale) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const float less = -1032.0f * scale;
  uint32_t magic = 0x64006400u;
  asm("" : "+v"(magic));  // in a vector register: an instruction takes one constant of another kind
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const f16x2 v = __builtin_bit_cast(f16x2, ((codes >> (4 * p)) & 0x000f000fu) | magic);
    r[p] = bf16_pair(__builtin_fmaf((float)v[0], scale, less), __builtin_fmaf((float)v[1], scale, less));
  }
  return __builtin_bit_cast(bf16x8, r);
}

// ---- few rows an expert

// The expert that a block of the few-rows kernel works on: `which`, or, where a batch (or band) has
// fewer rows than experts, that of row `which` if it is the expert's first (else no rows).  Its
// offsets come out of the lanes that searched for it, not of further loads that wait for the first.
struct Rows {
  int e, first, count;
};
__device__ __forceinline__ Rows few_rows_of(const ExpertDims& x, const int32_t* off, int which) {
  Rows r{which, 0, 0};
  if (x.rows >= x.E) {
    r.first = off[which];
    r.count = off[which + 1] - r.first;
    return r;
  }
  const int lane = threadIdx.x % kWave;
  const int step = (x.E + kWave - 1) / kWave;
  const int e1 = lane * step;
  const int start = off[0], v1 = off[min(e1, x.E)], total = off[x.E];
  const int row = start + which;
  // Lane 0 is in; the last lane in has the expert, or the first of its `step` candidates.
  const int at = __popcll(__ballot(e1 < x.E && v1 <= row)) - 1;
  int next;
  if (step == 1) {
    r.e = at;
    r.first = __builtin_amdgcn_readlane(v1, at);
    next = at + 1 < kWave ? __builtin_amdgcn_readlane(v1, min(at + 1, kWave - 1)) : total;
  } else {
    const int e2 = at * step + lane, v2 = off[min(e2, x.E)];
    const int in = __popcll(__ballot(lane < step && e2 < x.E && v2 <= row)) - 1;
    r.e = at * step + in;
    r.first = __builtin_amdgcn_readlane(v2, in);
    next = __builtin_amdgcn_readlane(v2, in + 1);  // step <= 16
  }
  if (r.first == row) r.count = next - row;
  return r;
}

// A strip is 16 columns of y with a gated activation (16 weight rows of the gate and 16 of the up
// projection), else 32.  A block of eight waves works for one expert, on R of its rows at a time,
// whose x it holds in LDS (the contraction in phases where it does not fit).  A wave, or `split` of
// them that share the contraction and add their parts through LDS in a fixed order, computes a
// strip: it loads codes and scales straight into registers, 1024 consecutive bytes a load, one
// step of U blocks of 128 ahead of the one that it multiplies.
//
// E2M1 weights are exact in bf16, scale and all.  INT4: the sums of a group's products with 128 + c
// and with -136 are added up in float32, which leaves the sum with c - 8, and the scale multiplies
// that sum: no weight is rounded.
template <int G, bool E2M1, int MT>
struct FewRows {
  static constexpr int kGroups = 128 / G;  // scales of a row and block
  static constexpr int U = !E2M1 && G == 32 ? 1 : 2;
  static constexpr int kWaves = 8;
  // LDS: two blocks a CU with 16 rows, one with 32.
  static constexpr int kPart = MT * 2 * 256;  // floats of a wave's results
  static constexpr int kLds = MT * 80 * 1024;
  static constexpr int kXBytes = kLds - kWaves * kPart * 4;

  // Codes and scales of U blocks of a strip.
  struct Step {
    u32x4 codes[U][2];
    u32x2 si[E2M1 ? 1 : U][2][kGroups];  // INT4: the scales of the lane's four result columns, a
                                         // column's groups side by side
    uint32_t se[E2M1 ? U : 1][2];        // E2M1: those of the lane's weight row
    // Scale of result column c for group q of block u.
    __device__ __forceinline__ float scale(int u, int h, int c, int q) const {
      const int at = c * kGroups + q;
      const uint32_t v = si[u][h][at / 4][at / 2 % 2];
      return __uint_as_float(at % 2 ? v & 0xffff0000u : v << 16);
    }
  };
};

// How a launch cuts its work.
struct FewSplit {
  int rows;    // R: rows of x in LDS
  int phase;   // blocks of 128 a phase
  int phases;
  int split;   // waves a strip
  int shares;  // blocks an expert
};

template <int G, bool E2M1, int MT, bool GATED>
__global__ __launch_bounds__(512, MT == 1 ? 4 : 2) void expert4_few_rows_kernel(
    ExpertDims x, Weights4 w4, FewSplit cut, const int32_t* __restrict__ off,
    const char* __restrict__ a, const char* __restrict__ codes, const char* __restrict__ scales,
    const float* __restrict__ bias, const uint16_t* __restrict__ residual, uint16_t* __restrict__ y,
    int strips, uint32_t base) {
  using F = FewRows<G, E2M1, MT>;
  using Step = typename F::Step;
  constexpr int U = F::U, kGroups = F::kGroups;
  constexpr int kCols = GATED ? 16 : 32;  // columns of y a strip
  __shared__ __align__(1024) char lds[F::kLds];
  float* part = reinterpret_cast<float*>(lds + F::kXBytes);  // [kWaves][kPart]
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t block = base + blockIdx.x;  // below 2^26
  const Rows of = few_rows_of(x, off, (int)(block / (uint32_t)cut.shares));
  const int e = of.e, o0 = of.first, rows = of.count;
  if (rows <= 0) return;
  const int strip = (int)(block % (uint32_t)cut.shares) * (F::kWaves / cut.split) + wave / cut.split;
  const int member = wave % cut.split;
  const uint32_t ld = (uint32_t)x.K * 2;
  const int i = lane & 15, g = lane >> 4;
  const uint32_t codes_bytes = w4.tiles * w4.codes_stride(), scales_bytes = w4.tiles * w4.scales_stride();
  const __amdgpu_buffer_rsrc_t rw = uniform_buffer(codes + (int64_t)e * codes_bytes, codes_bytes);
  const __amdgpu_buffer_rsrc_t rs = uniform_buffer(scales + (int64_t)e * scales_bytes, scales_bytes);
  bf16x8 offset;
#pragma unroll
  for (int q = 0; q < 8; ++q) offset[q] = (__bf16)-kInt4Offset;

  // A place in the wave's work: the phase, and blocks [block, last) that are left of its part of it.
  struct Cursor {
    int phase, block, last;
  };
  auto enter = [&](Cursor& c) {
    const int p0 = c.phase * cut.phase, n = min(cut.phase, w4.blocks - p0);
    c.block = p0 + member * n / cut.split;
    c.last = p0 + (member + 1) * n / cut.split;
  };
  auto load = [&](Step& t, const Cursor& c) {
    if (c.phase >= cut.phases || strip >= strips) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (The 16 rows are one tile, or the halves of two where an expert's up projection starts at
      // an odd multiple of 8.  Rows past the last give results that are not stored, or are past the
      // descriptor's end.)
      const uint32_t row = (uint32_t)strip * kCols + h * (GATED ? x.N : 16);
      const uint32_t r = row + i, q4 = row + g * 4;
      const uint32_t vw = (r >> 4) * w4.codes_stride() + ((r & 15) | g << 4) * 16;
      const uint32_t vs = E2M1 ? (r >> 4) * w4.scales_stride() + (r & 15) * 4
                               : (q4 >> 4) * w4.scales_stride() + (q4 & 15) * kGroups * 2;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t b = (uint32_t)min(c.block + u, c.last - 1);  // (past the end: not multiplied)
        t.codes[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, vw + b * 1024, 0, 0);
        if constexpr (E2M1) {
          t.se[u][h] = __builtin_amdgcn_raw_buffer_load_b32(rs, vs + b * 64, 0, 0);
        } else if constexpr (kGroups == 1) {
          t.si[u][h][0] = __builtin_amdgcn_raw_buffer_load_b64(rs, vs + b * 32, 0, 0);
        } else {
#pragma unroll
          for (int q = 0; q < kGroups; q += 2) {
            const u32x4 v =
                __builtin_amdgcn_raw_buffer_load_b128(rs, vs + b * (kGroups * 32) + q * 8, 0, 0);
            t.si[u][h][q] = u32x2{v[0], v[1]};
            t.si[u][h][q + 1] = u32x2{v[2], v[3]};
          }
        }
      }
    }
  };
  // Waits for the wave's own LDS accesses, then for the block's other waves (and not for the
  // loads under way).
  auto meet = []() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  // x in LDS: rows of cut.phase blocks of 16 chunks (16 bytes), chunk c of row r at c ^ r (of the
  // lower four bits), so that the 16 rows of a read fall into different banks.
  const uint32_t row_bytes = (uint32_t)cut.phase * 256;
  uint32_t from[4];  // of the lane's fragments s of block 0, rows i
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = min(i, cut.rows - 1);  // (lanes of absent rows: results that are not stored)
    from[s] = r * row_bytes + (((s * 4 + g) ^ (r & 15)) << 4);
  }

  for (int r0 = 0; r0 < rows; r0 += cut.rows) {
    const int here = min(rows - r0, cut.rows);
    auto stage = [&](int phase) {
      const int k0 = phase * cut.phase * 128;
      const int segments = (min(cut.phase, w4.blocks - phase * cut.phase) + 3) / 4;  // of 64 chunks
      const char* src = a + (int64_t)(o0 + r0) * ld + (int64_t)k0 * 2;
      constexpr int kAhead = 4;
      for (int q0 = wave; q0 < here * segments; q0 += F::kWaves * kAhead) {
        u32x4 v[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int q = q0 + n * F::kWaves, row = q / segments, c = q % segments * 64 + lane;
          v[n] = u32x4{0, 0, 0, 0};  // chunks past the row's end
          if (q < here * segments && k0 + c * 8 < x.K)
            v[n] = *reinterpret_cast<const u32x4*>(src + (int64_t)row * ld + c * 16);
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int q = q0 + n * F::kWaves, row = q / segments, c = q % segments * 64 + lane;
          if (q < here * segments && c < cut.phase * 16)
            *reinterpret_cast<u32x4*>(lds + row * row_bytes + ((c ^ (row & 15)) << 4)) = v[n];
        }
      }
    };
    f32x4 acc[MT][2];
    auto multiply = [&](const Step& t, const Cursor& c) {
      const char* xs = lds + (c.block - c.phase * cut.phase) * 256;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u > 0 && c.block + u >= c.last) break;
        auto fragment = [&](int s, int m) {
          return *reinterpret_cast<const bf16x8*>(xs + from[s] + m * 16 * row_bytes + u * 256);
        };
        if constexpr (E2M1) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            bf16x8 fx[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) fx[m] = fragment(s, m);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bf16x8 f = decode_e2m1(t.codes[u][h][s], e2m1_scale((t.se[u][h] >> (8 * s)) & 0xffu));
#pragma unroll
              for (int m = 0; m < MT; ++m)
                acc[m][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, fx[m], acc[m][h], 0, 0, 0);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < kGroups; ++q) {
            f32x4 sum[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) sum[m][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            bf16x8 fx[G / 32][MT];
#pragma unroll
            for (int s = 0; s < G / 32; ++s)
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                fx[s][m] = fragment(q * (G / 32) + s, m);
                sum[m][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(offset, fx[s][m], sum[m][0], 0, 0, 0);
              }
#pragma unroll
            for (int m = 0; m < MT; ++m) sum[m][1] = sum[m][0];
#pragma unroll
            for (int s = 0; s < G / 32; ++s)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const bf16x8 f = decode_int4(t.codes[u][h][q * (G / 32) + s]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  sum[m][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, fx[s][m], sum[m][h], 0, 0, 0);
              }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int c4 = 0; c4 < 4; ++c4) {
                const float scale = t.scale(u, h, c4, q);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  acc[m][h][c4] = __builtin_fmaf(scale, sum[m][h][c4], acc[m][h][c4]);
              }
            }
            __builtin_amdgcn_sched_barrier(0);  // else all reads come first, and registers run out
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // acc[m][h][q]: column g * 4 + q of half h of the strip, row m * 16 + i.
    auto finish = [&]() {
      if (cut.split > 1) {
        if (member > 0) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<f32x4*>(part + wave * F::kPart + (m * 2 + h) * 256 + lane * 4) = acc[m][h];
        }
        meet();
        if (member == 0) {
          for (int q = 1; q < cut.split; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                acc[m][h] += *reinterpret_cast<const f32x4*>(part + (wave + q) * F::kPart +
                                                             (m * 2 + h) * 256 + lane * 4);
        }
        meet();
      }
      if (member > 0 || strip >= strips) return;
      const int col = strip * kCols + g * 4;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m * 16 + i >= here) continue;
        const int64_t row = o0 + r0 + m * 16 + i;
        float z[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = GATED ? col : col + h * 16;
          f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
          if (bias != nullptr && c < x.N)
            b = *reinterpret_cast<const f32x4*>(bias + (int64_t)e * x.Z + (GATED ? h * x.N : 0) + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) z[h][q] = acc[m][h][q] + b[q];
        }
        float out[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) out[q] = GATED ? (q < 4 ? z[0][q] : 0.0f) : z[q / 4][q % 4];
        act_values(x.act, out);
#pragma unroll
        for (int h = 0; h < (GATED ? 1 : 2); ++h) {
          const int c = col + h * 16;
          if (c >= x.N) continue;
          float* o = out + h * 4;
          if constexpr (GATED) {
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] *= z[1][q];
          }
          if (residual != nullptr) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(residual + row * x.N + c);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              o[2 * q] += __uint_as_float(v[q] << 16);
              o[2 * q + 1] += __uint_as_float(v[q] & 0xffff0000u);
            }
          }
          *reinterpret_cast<u32x2*>(y + row * x.N + c) = u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
        }
      }
    };

    // Two steps at a time, the next one's loads under the products of each.
    Step even, odd;
    Cursor now{0, 0, 0};
    enter(now);
    load(even, now);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc[m][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int phase = 0; phase < cut.phases; ++phase) {
      meet();  // what is there has been read
      stage(phase);
      meet();
      if (strip >= strips) continue;
      while (now.phase == phase) {
        Cursor second = now;
        second.block += U;
        const bool two = second.block < now.last;
        if (two) load(odd, second);
        __builtin_amdgcn_sched_barrier(0);
        multiply(even, now);
        Cursor next = second;
        next.block += U;
        if (next.block >= next.last) {
          ++next.phase;
          enter(next);
        }
        load(even, next);
        __builtin_amdgcn_sched_barrier(0);
        if (two) multiply(odd, second);
        now = next;
      }
    }
    finish();
  }
}

// ---- many rows an expert

// A block computes tiles of BM rows x 256 columns, one after another, as the products of bf16
// weights do (the order of the tiles, of a wave's rows and columns, and the epilogue are the same).
// x goes straight to LDS, in stages of 64 along the contraction, three deep.  The weights do not
// pass through LDS: a wave loads the codes of its own 64 columns into registers, a block of 128 along
// the contraction ahead (a fourth of what bf16 takes), and turns eight codes a lane and fragment
// into bf16 while the products of the step before run.
template <int G, bool E2M1, bool GATED_>
struct Tile4 {
  static constexpr int WM = 1, WN = 4, BM = 128, BN = 256, MI = 8, NJ = 4;
  static constexpr bool GATED = GATED_;
  static constexpr int kNW = WM * WN, kThreads = kNW * kWave;
  static constexpr int kHalf = BM * 64;      // bytes of 32 along the contraction
  static constexpr int kStage = 2 * kHalf, kStages = 3, kLds = kStages * kStage;
  static constexpr int QA = kStage / 1024 / kNW;  // loads a wave and stage
  static constexpr int kQuarter = BM / 4;
  static constexpr int kGroups = 128 / G;         // scales of a row and block
  static constexpr int kScaleBytes = kGroups * (E2M1 ? 1 : 2);
  static constexpr int kPacked = 2 * NJ;         // loads of codes and scales a wave and block

  // Codes and scales of a block of 128 of the wave's columns.
  struct Packed {
    u32x4 codes[NJ];
    uint32_t scales[NJ][(kScaleBytes + 3) / 4];
  };
  // What is loaded next: a block of 128 of a tile.
  struct Cursor {
    const char *a, *codes, *scales;            // the tile's first row; the expert's weights
    uint32_t a_bytes, codes_bytes, scales_bytes;
    int n0;                                    // the tile's first column of y
    int block;
  };

  f32x4 acc[MI][NJ];
  uint32_t va[QA];     // byte offsets of this lane's loads of a stage
  uint32_t lda, codes_stride, scales_stride;
  char* lds;
  int wave, lane, K, blocks, second;
  int at;              // byte offset of the lane's part of a half stage's first fragment
  int put;             // LDS offset of the stage that is read next
  static constexpr int m0 = 0;  // every wave has all the rows of the tile

  __device__ __forceinline__ Tile4(char* lds_, const ExpertDims& x, const Weights4& w4)
      : lda((uint32_t)x.K * 2), codes_stride(w4.codes_stride()), scales_stride(w4.scales_stride()),
        lds(lds_), K(x.K), blocks(w4.blocks), second(x.N), put(0) {
    lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    at = (lane & 15) * 64 + (((lane >> 4) ^ swizzle(lane & 15)) << 4);
#pragma unroll
    for (int q = 0; q < QA; ++q)
      va[q] = (uint32_t)((q % 2 * kNW + wave) * 16 + lane / 4) * lda + chunk() * 16 + q / 2 * 64;
    static_assert(QA == 4 && BM / 16 == 2 * kNW);
  }

  // LDS row r of a half stage (64 bytes) holds chunk p ^ swizzle(r) at position p.
  static __device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 3; }
  __device__ __forceinline__ int chunk() const { return (lane & 3) ^ swizzle(lane / 4); }

  // Codes and scales of the cursor's block.  Fragment j of a wave has the columns 32 (j / 2) + 8 g +
  // 4 (j % 2) + 0..3 of its 64 in lane group g of the results (of the gate for j < 2 and of the up
  // projection else, where gated), so lane i of the operand has the weight row of the column with
  // g = i / 4 and i % 4.
  __device__ __forceinline__ void load_packed(Packed& p, const Cursor& c) const {
    const __amdgpu_buffer_rsrc_t rw = uniform_buffer(c.codes, c.codes_bytes);
    const __amdgpu_buffer_rsrc_t rs = uniform_buffer(c.scales, c.scales_bytes);
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = c.n0 + wave % WN * (GATED ? 32 : 64) + i / 4 * 8 + j % 2 * 4 + i % 4;
      const uint32_t r = (uint32_t)(col + j / 2 * (GATED ? second : 32));
      p.codes[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rw, (r >> 4) * codes_stride + c.block * 1024 + ((r & 15) | g << 4) * 16, 0, 0);
      const uint32_t vs = (r >> 4) * scales_stride + (c.block * 16 + (r & 15)) * kScaleBytes;
      if constexpr (kScaleBytes == 2) {
        p.scales[j][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, vs, 0, 0);
      } else if constexpr (kScaleBytes == 4) {
        p.scales[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, vs, 0, 0);
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, vs, 0, 0);
        p.scales[j][0] = v[0];
        p.scales[j][1] = v[1];
      }
    }
  }

  // Loads half `h` of the cursor's block of x into the stage at `to`.
  __device__ __forceinline__ void load_x(const Cursor& c, int h, char* to) const {
    const int done = c.block * 128 + h * 64;
    const __amdgpu_buffer_rsrc_t r = uniform_buffer(
        c.a + (int64_t)done * 2, c.a_bytes > (uint32_t)done * 2 ? c.a_bytes - (uint32_t)done * 2 : 0);
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      // Chunks past the end of the contraction read as zeros.
      const bool in = done + q / 2 * 32 + chunk() * 8 < K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void*)(to + (q * kNW + wave) * 1024), 16,
                                               in ? va[q] : kPast, 0, 0, 0);
    }
  }

  // Fragment j of step s (32 along the contraction) of a block.
  static __device__ __forceinline__ bf16x8 decode(const Packed& p, int j, int s) {
    if constexpr (E2M1) {
      return decode_e2m1(p.codes[j][s], e2m1_scale((p.scales[j][0] >> (8 * s)) & 0xffu));
    } else {
      const int q = s * 32 / G;
      const uint32_t v = p.scales[j][q / 2];
      return decode_int4_scaled(p.codes[j][s], __uint_as_float(q % 2 ? v & 0xffff0000u : v << 16));
    }
  }

  static __device__ __forceinline__ int stage_after(int at) {
    return at == (kStages - 1) * kStage ? 0 : at + kStage;
  }

  // Waits until none of this wave's LDS reads and at most N (< 0: any number) of its loads are
  // under way, then for the block's other waves.
  template <int N>
  static __device__ __forceinline__ void wait_and_meet() {
    if constexpr (N < 0)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // One step of 32: products of the fragments b with x at `from`, and the fragments of step S of p.
  // rows: rows of the tile that there are (the products of absent quarters are skipped).
  template <int S>
  __device__ __forceinline__ void step(const char* from, int rows, const bf16x8 (&b)[NJ],
                                       bf16x8 (&then)[NJ], const Packed& p) {
    const char* mine = from + at;
    auto read = [&](int m) { return *reinterpret_cast<const bf16x8*>(mine + m * 1024); };
    bf16x8 a[2][2] = {{read(0), read(1)}, {}};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q < 3) {
        a[(q + 1) % 2][0] = read(2 * q + 2);
        a[(q + 1) % 2][1] = read(2 * q + 3);
      }
      if (q == 0 || rows > q * kQuarter) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[2 * q + m][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[q % 2][m], acc[2 * q + m][j], 0, 0, 0);
      }
      then[q] = decode(p, q, S);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Half of a block: its two steps, under the loads of the same half of the cursor's block.  The two
  // stages are different ones, and saying so (restrict) keeps the reads from waiting for the loads.
  template <int H>
  __device__ __forceinline__ void half(const Cursor& c, char* __restrict__ to,
                                       const char* __restrict__ from, int rows, bf16x8 (&b)[NJ],
                                       const Packed& now, const Packed& then) {
    load_x(c, H, to);
    bf16x8 f[NJ];
    step<2 * H + 1>(from, rows, b, f, now);
    step<H == 0 ? 2 : 0>(from + kHalf, rows, f, b, H == 0 ? now : then);
  }

  // acc = x w^T of a tile.  now: its first block's codes, b: the fragments of its first step; both
  // are the next tile's afterwards.  next(cursor) sets the cursor to the block after.
  // Order of a wave's loads: a block's codes and scales, its first half of x, its second half; a
  // half is waited for one half before the next is asked for.
  template <typename Next>
  __device__ __forceinline__ void run(Cursor& c, const Next& next, int rows, Packed& now,
                                      bf16x8 (&b)[NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int n = 0; n < blocks; ++n) {
      // The tile's first block had landed before the last epilogue.
      if (n == 0)
        wait_and_meet<-1>();
      else
        wait_and_meet<QA>();
      Packed then;
      load_packed(then, c);
      const int second_half = stage_after(put), free = stage_after(second_half);
      half<0>(c, lds + free, lds + put, rows, b, now, then);
      if (n == 0)
        wait_and_meet<-1>();
      else
        wait_and_meet<QA + kPacked>();
      half<1>(c, lds + put, lds + second_half, rows, b, now, then);
      put = free;
      now = then;
      next(c);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
};

template <typename P>
__global__ __launch_bounds__(P::kThreads, 2) void expert4_rows_kernel(
    ExpertDims x, Weights4 w4, const int32_t* __restrict__ off, const char* __restrict__ a,
    const char* __restrict__ codes, const char* __restrict__ scales, const float* __restrict__ bias,
    const uint16_t* __restrict__ residual, uint16_t* __restrict__ y, int ntiles) {
  __shared__ __align__(1024) char lds[P::kLds + sizeof(RowTiles)];
  RowTiles& table = *reinterpret_cast<RowTiles*>(lds + P::kLds);
  constexpr int kCols = P::GATED ? P::BN / 2 : P::BN;  // columns of y a tile
  table.build<P::BM, P::kThreads>(off, x.E);
  const TileGrid<P::BM, P::BN> grid(1, __builtin_amdgcn_readfirstlane(table.first[x.E]), ntiles);
  const int numbers = grid.numbers();
  const uint32_t ld = (uint32_t)x.K * 2;
  int number = blockIdx.x;
  Segment ahead{0, 0, 0};
  const uint32_t codes_bytes = w4.tiles * w4.codes_stride(), scales_bytes = w4.tiles * w4.scales_stride();
  typename P::Cursor c{a, codes, scales, 0, 0, 0, 0, -1};
  // The block after the cursor's: at a tile's end the first of the next tile, if there is one (else
  // of none: it loads nothing).
  auto next = [&](typename P::Cursor& c) {
    if (c.block >= 0 && ++c.block < w4.blocks) return;
    c = {a, codes, scales, 0, 0, 0, 0, 0};
    ahead.rows = 0;
    for (; number < numbers; number += gridDim.x) {
      const Tile t = grid.at(number);
      if (!t.live) continue;
      const Segment s = ahead = segment_of<P::BM>(table, off, x.E, t.m);
      c.a = a + (int64_t)s.row * ld;
      c.a_bytes = (uint32_t)s.rows * ld;
      c.codes = codes + (int64_t)s.e * codes_bytes;
      c.scales = scales + (int64_t)s.e * scales_bytes;
      c.codes_bytes = codes_bytes;
      c.scales_bytes = scales_bytes;
      c.n0 = t.n * kCols;
      number += gridDim.x;
      break;
    }
  };
  next(c);
  if (ahead.rows <= 0) return;
  P p(lds, x, w4);
  typename P::Packed packed;
  bf16x8 b[P::NJ];
  p.load_packed(packed, c);
  p.load_x(c, 0, lds);
  p.load_x(c, 1, lds + P::kStage);
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) b[j] = P::decode(packed, j, 0);
  Segment s = ahead;
  int col0 = c.n0;
  next(c);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  while (s.rows > 0) {
    Segment loaded = ahead;  // tile of the block that was loaded last: after run the next tile
    int loaded_col0 = c.n0;
    auto step = [&](typename P::Cursor& q) {
      loaded = ahead;
      loaded_col0 = q.n0;
      next(q);
    };
    p.run(c, step, s.rows, packed, b);

    const int g = p.lane >> 4;
    const int c0 = col0 + p.wave % P::WN * (P::GATED ? 32 : 64) + g * 8;
    float bz[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) bz[q] = 0.0f;
    if (bias != nullptr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = P::GATED ? c0 : c0 + h * 32;
        if (col < x.N) {
          const f32x4* q = reinterpret_cast<const f32x4*>(bias + (int64_t)s.e * x.Z + col +
                                                          (P::GATED ? h * x.N : 0));
          const f32x4 lo = q[0], hi = q[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bz[h * 8 + i] = lo[i];
            bz[h * 8 + 4 + i] = hi[i];
          }
        }
      }
    }
    rows_epilogue<P, 0>(p, x, s, c0, bz, residual, y, nullptr);
    rows_epilogue<P, 4>(p, x, s, c0, bz, residual, y, nullptr);
    s = loaded;
    col0 = loaded_col0;
  }
}

// The kernel for few rows is taken up to 20 rows an expert on average, and up to 96 where the tiles
// would leave half of the CUs without one.  Its passes take 16 rows where no expert has more or
// they have up to 12 on average, else 32.  In us, passes of 16, of 32, and tiles, INT4 in groups of
// 128 (E2M1): 64 experts, top-8, 2048 -> 2 x 1024: 16 tokens 26, 35, 48 (24, 28, 35), 64 tokens 34,
// 39, 48, 128 tokens 47, 41, 48 (42, 35, 38), 256 tokens 72, 69, 55 (66, 56, 44); 30 experts, top-2,
// 4096 -> 4096: 128 tokens 64, 74, 91, 256 tokens 95, 77, 90, 512 tokens 143, 135, 102; 8 experts of
// those: 256 tokens 85, 66, 84, 512 tokens 146, 108, 92.
bool few4(const ExpertDims& x) {
  const int tiles = ceil_div(x.N, gated(x.act) ? 128 : 256);
  return x.T <= 32 || (int64_t)x.rows <= (int64_t)x.E * 20 ||
         ((int64_t)x.rows <= (int64_t)x.E * 96 && (int64_t)x.E * tiles <= kCus / 2);
}

hipError_t expert_rows4(const ExpertDims& x, const Weights4& w4, const int32_t* off,
                        const uint16_t* a, const void* packed, const float* bias,
                        const uint16_t* residual, uint16_t* y, hipStream_t s) {
  const char* codes = static_cast<const char*>(packed);
  const char* scales = codes + w4.codes_bytes();
  auto by_rows = [&](auto group, auto e2m1) {
    constexpr int G = decltype(group)::value;
    constexpr bool E2M1 = decltype(e2m1)::value;
    auto few = [&](auto tiles) {
      constexpr int MT = decltype(tiles)::value;
      using F = FewRows<G, E2M1, MT>;
      const int strips = ceil_div(x.N, gated(x.act) ? 16 : 32);
      const int experts = std::min(x.E, x.rows);
      FewSplit cut{};
      cut.rows = MT * 16;
      if (MT == 1) {
        // Fewer rows at a time where the contraction is too long for 16 and experts have few.
        const int wanted = 2 * ceil_div(x.rows, x.E) + 2;
        while (cut.rows > 4 && cut.rows * w4.blocks * 256 > F::kXBytes &&
               (cut.rows / 2 >= x.T || cut.rows / 2 >= wanted))
          cut.rows /= 2;
      }
      cut.phase = std::min(w4.blocks, F::kXBytes / (cut.rows * 256));
      cut.phases = ceil_div(w4.blocks, cut.phase);
      cut.phase = ceil_div(w4.blocks, cut.phases);  // about equal ones
      const int least = w4.blocks - (cut.phases - 1) * cut.phase;  // blocks of the last phase
      const int64_t units = (int64_t)experts * strips;
      // Waves share strips until there are eight a CU.  In us with 1, 2, 4 and 8 waves a strip: one
      // token of top-8, 2048 -> 2 x 1024 (512 strips) 13.8, 9.6, 7.8, 8.5; 7168 -> 2 x 1024 35.8, 21.4,
      // 14.9, 15.8; 4 tokens of the former (1600) 15.6, 16.5, 17.4, 22.2.
      cut.split = 1;
      while (cut.split < 8 && cut.split * 2 <= least && units * cut.split < kCus * 8) cut.split *= 2;
      cut.shares = ceil_div(strips, F::kWaves / cut.split);
      return in_ranges((int64_t)experts * cut.shares, [&](dim3 blocks, int64_t b) {
        return launch(MOE_KERNEL_EXPERT4_FEW_ROWS,
                      gated(x.act) ? expert4_few_rows_kernel<G, E2M1, MT, true>
                                   : expert4_few_rows_kernel<G, E2M1, MT, false>,
                      blocks, dim3(F::kWaves * kWave), 0, s, x, w4, cut, off,
                      reinterpret_cast<const char*>(a), codes, scales, bias, residual, y, strips, b);
      });
    };
    auto tiles = [&](auto tile) {
      using P = typename decltype(tile)::type;
      const int ntiles = ceil_div(x.N, P::GATED ? P::BN / 2 : P::BN);
      return launch(MOE_KERNEL_EXPERT4_ROWS, expert4_rows_kernel<P>, row_blocks<P>(x, ntiles),
                    dim3(P::kThreads), 0, s, x, w4, off, reinterpret_cast<const char*>(a), codes, scales,
                    bias, residual, y, ntiles);
    };
    if (few4(x)) {
      if (x.T <= 16 || (int64_t)x.rows <= (int64_t)x.E * 12) return few(std::integral_constant<int, 1>());
      return few(std::integral_constant<int, 2>());
    }
    return gated(x.act) ? tiles(Type<Tile4<G, E2M1, true>>()) : tiles(Type<Tile4<G, E2M1, false>>());
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
