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

// Eight INT4 codes c (0..15) as the bf16 numbers 16 + c: the code is the upper four bits of the mantissa
// under the exponent of 16.  (As the lower four, under that of 128, a group's sums are of six times the
// magnitude, and lose that much more to rounding.)  One rotation and one mask with the exponent for a
// pair, none for the first.
constexpr float kInt4Offset = 24.0f;  // 16 + c stands for c - 8
__device__ __forceinline__ bf16x8 decode_int4(uint32_t codes) {
  uint32_t magic = 0x41804180u;
  asm("" : "+v"(magic));  // in a vector register: an instruction takes one constant of another kind
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    r[p] = (__builtin_rotateright32(codes, 4 * p) & 0x00780078u) | magic;
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

// INT4 scales of four consecutive weight rows, for a block of 128 along the contraction.
template <int G>
struct Int4Scales {
  static constexpr int kGroups = 128 / G;
  static constexpr int kRow = kGroups == 1 ? 2 : 4;  // bytes of a row's scales that are side by side
  u32x4 v[(kGroups + 1) / 2];
  // Those of groups q and q + 1 (of the only one); at: where the first row's for the block are.
  __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& from, uint32_t at, int q) {
    if constexpr (kGroups == 1) {
      const u32x2 r = __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, 0);
      v[0][0] = r[0];
      v[0][1] = r[1];
    } else {
      v[q / 2] = __builtin_amdgcn_raw_buffer_load_b128(from, at + q * 32, 0, 0);
    }
  }
  // That of row r (0..3) for group q.
  __device__ __forceinline__ float get(int r, int q) const {
    const uint32_t w = kGroups == 1 ? v[0][r / 2] : v[q / 2][r];
    return __uint_as_float((kGroups == 1 ? r : q) % 2 ? w & 0xffff0000u : w << 16);
  }
};

// A strip is 16 columns of y with a gated activation (16 weight rows of the gate and 16 of the up
// projection), else 32.  A block of eight waves works for one expert, on R of its rows at a time,
// whose x it holds in LDS (the contraction in phases where it does not fit).  A wave, or `split` of
// them that share the contraction and add their parts through LDS in a fixed order, computes a
// strip: it loads codes and scales straight into registers, 1024 consecutive bytes a load, one
// step of U blocks of 128 ahead of the one that it multiplies.
//
// E2M1 weights are exact in bf16, scale and all.  INT4: the sums of a group's products with 16 + c
// and with -24 are added up in float32, which leaves the sum with c - 8, and the scale multiplies
// that sum: no weight is rounded.
//
// Bound by HBM.  16 tokens, top-8 of 64, 2048 -> 2 x 1024, E2M1: 26 us, 5 TB/s of codes and scales (INT4
// in groups of 128, 64 and 32: 30, 33, 34); of 256 experts, 7168 -> 2 x 1024, INT4 in groups of 128: 149
// us, 5.2 TB/s (64 and 32: 170, 193); one token of the former 7.4 us, a launch and the chain offsets ->
// codes -> products -> join.  x in registers instead of LDS spilled and halved the waves; several
// strips a wave, one after another, and passes of 64 rows were slower.  For 16 rows and groups of 64
// and 32 some registers spill: 8 and 16 bytes of scratch a lane, 36 and 40 with a gate.
//
// Skewed routing: a busy expert's passes follow one another in its blocks.  190 tokens, top-8 of 256,
// 2048 -> 2 x 1024, take 117 us with uniform routing (13 rows at most) and 143 under Zipf 1.2 with 0.7 of
// the weights (186 rows: twelve passes).
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
    Int4Scales<G> si[E2M1 ? 1 : U][2];  // INT4: those of the lane's four result columns
    uint32_t se[E2M1 ? U : 1][2];       // E2M1: those of the lane's weight row
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
                               : (q4 >> 4) * w4.scales_stride() + (q4 & 15) * Int4Scales<G>::kRow;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t b = (uint32_t)min(c.block + u, c.last - 1);  // (past the end: not multiplied)
        t.codes[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, vw + b * 1024, 0, 0);
        if constexpr (E2M1) {
          t.se[u][h] = __builtin_amdgcn_raw_buffer_load_b32(rs, vs + b * 64, 0, 0);
        } else {
#pragma unroll
          for (int q = 0; q < kGroups; q += 2) t.si[u][h].load(rs, vs + b * (kGroups * 32), q);
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
                const float scale = t.si[u][h].get(c4, q);
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

// A block computes tiles of 64 or 128 rows x 256 columns, one after another, as the products of bf16
// weights do (the order of the tiles, of a wave's rows and columns, and the epilogue are the same).
// x goes straight to LDS, in stages of 128 along the contraction.  The weights do not pass through
// LDS: a wave loads the codes of its own 64 columns into registers, a block of 128 along the
// contraction ahead (a fourth of what bf16 takes), and turns eight codes a lane and fragment into
// bf16 between the products; what runs beside them is the other block of the CU.
//
// INT4: no weight is rounded.  A group's products with 16 + c are added up in sums of their own,
// which start from its products with -24 and so come to those with c - 8, and the scale multiplies
// the finished sums into the accumulators.  The products with -24 are the same for all columns: each
// of the four waves computes them for a quarter of the rows, of the next block, and leaves them in
// LDS (with each computing all of them: 591 us against 580 for 8 experts, top-2, 8192 tokens, 4096 ->
// 4096).  A wave takes 16 rows x 64 columns at a time through a group, whose fragments it has
// expanded, so that the sums take 16 registers; tiles of 64 rows leave room for them.  With 128 rows
// registers run out (425 us for 64 experts, top-8, 4096 tokens, 2048 -> 2 x 1024, against 355), and
// with groups of 32, whose scales take a quarter of the registers, they do with 64 rows too (3200 us;
// the kernel for few rows takes 740).  Without a branch after every 16 rows the scaling of one 16 runs
// under the products of the next: 332 us and 537 for the two, but 43 against 41 for 256 tokens of the
// first, which is for experts of 96 rows and more on average, and for groups of 128 (of 64: registers
// run out).
//
// E2M1 weights are bf16 numbers, scale and all.  Tiles of 128 rows where there are four a CU and
// experts have that many: 253 us for the 4096 tokens, 450 for the 8192 (266 and 464 with branches),
// against 314 and 514 with 64 rows, which leave fewer products for each weight that is expanded; where
// there are fewer tiles, 64 rows: 68 us against 82 for 512 tokens of the latter, 27 against 33 for
// 1021 tokens, top-4 of 30, 776 -> 1000.
//
// What bounds the large products: with INT4 the matrix cores are busy in 40% of the cycles and the
// vector units, which expand codes and scale sums, in as many, and little of the one runs under the
// other; a SIMD has room for two waves.  The loads take their part: the compiler issues those of the
// next codes and of x at the end of a block's products where they have no branches (after 112 of 128
// matrix instructions in E2M1 tiles of 128 rows, 50 to 54 of 64 in INT4 ones), and ahead of them where
// they have; and in INT4 tiles it waits for all of them before it reads x for the products with -24,
// since it cannot tell the stages of LDS apart, so that of the blocks of x under way (kAhead) the
// next one's latency shows.
template <int G, bool E2M1, bool GATED_, int MI_, bool SKIP>
struct Tile4 {
  static constexpr int WM = 1, WN = 4, MI = MI_, BM = MI * 16, BN = 256, NJ = 4;
  static constexpr bool GATED = GATED_;
  static constexpr int kNW = WM * WN, kThreads = kNW * kWave;
  static constexpr int kStage = BM * 256, kStages = MI == 8 ? 2 : E2M1 ? 3 : 4;
  static constexpr int kAhead = kStages - 1;      // blocks of x that are under way
  static constexpr int QA = kStage / 1024 / kNW;  // loads of x a wave and block
  static constexpr int kGroups = 128 / G;         // groups of a row and block
  static constexpr int kSteps = G / 32;           // matrix instructions a group and fragment
  static constexpr int m0 = 0;  // every wave has all the rows of the tile
  // INT4: a block's products with -24, [group][row] (four times each), of this block and the next.
  static constexpr int kLess = E2M1 ? 0 : kGroups * BM * 16;
  static constexpr int kLds = kStages * kStage + 2 * kLess;

  // Codes of a block of 128 of the wave's columns, and the scales of the lane's results.
  struct Packed {
    u32x4 codes[NJ];
    std::conditional_t<E2M1, uint32_t, Int4Scales<G>> scales[NJ];
  };
  // A place in the block's work: a tile, and a block of 128 of it.
  struct Walk {
    int number;   // of the tile after
    Segment s;    // the tile's rows (none: no tile is left)
    int n0;       // its first column of y
    int block;
  };

  f32x4 acc[MI][NJ];
  const char *x, *codes, *scales;
  uint32_t lda, codes_stride, scales_stride, codes_bytes, scales_bytes;
  int wave, lane, K, blocks, second;
  uint32_t va;       // byte offset of this lane's first load of a block of x
  uint32_t from_[4]; // byte offsets of the lane's fragments s of the first 16 rows of a stage
  int put;           // LDS offset of the stage that is read next
  int less;          // and of its products with -24
  bf16x8 offset;

  __device__ __forceinline__ Tile4(const ExpertDims& d, const Weights4& w4, const char* x_,
                                      const char* codes_, const char* scales_)
      : x(x_), codes(codes_), scales(scales_), lda((uint32_t)d.K * 2), codes_stride(w4.codes_stride()),
        scales_stride(w4.scales_stride()), codes_bytes(w4.tiles * w4.codes_stride()),
        scales_bytes(w4.tiles * w4.scales_stride()), K(d.K), blocks(w4.blocks), second(d.N), put(0),
        less(kStages * kStage) {
    lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int i = lane & 15, g = lane >> 4;
    va = (uint32_t)(wave * 4 + g) * lda + chunk() * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) from_[s] = i * 256 + (((s * 4 + g) ^ i) << 4);
#pragma unroll
    for (int q = 0; q < 8; ++q) offset[q] = (__bf16)-kInt4Offset;
  }

  // A stage has rows of 256 bytes, 16 chunks; position p of row r holds chunk p ^ r (of the lower
  // four bits).  A load of a wave takes four rows, row 16 q + 4 wave + lane / 16 for its q-th.
  __device__ __forceinline__ int chunk() const { return (lane & 15) ^ (wave * 4 + (lane >> 4)); }

  __device__ __forceinline__ void load_x(const Walk& w, char* to) const {
    const uint32_t done = (uint32_t)w.block * 256, bytes = (uint32_t)w.s.rows * lda;
    const __amdgpu_buffer_rsrc_t r =
        uniform_buffer(x + (int64_t)w.s.row * lda + done, bytes > done ? bytes - done : 0);
    // Chunks past the end of the contraction read as zeros.
    const bool in = w.block * 128 + chunk() * 8 < K;
#pragma unroll
    for (int q = 0; q < QA; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void*)(to + (q * kNW + wave) * 1024), 16,
                                               in ? va + q * 16 * lda : kPast, 0, 0, 0);
  }

  // Fragment j of a wave has the columns 32 (j / 2) + 8 g + 4 (j % 2) + 0..3 of its 64 in lane group g
  // of the results (of the gate for j < 2 and of the up projection else, where gated), so lane i of
  // the operand has the weight row of the column with g = i / 4 and i % 4.
  __device__ __forceinline__ int first_column(const Walk& w, int j) const {
    return w.n0 + wave * (GATED ? 32 : 64) + j % 2 * 4 + j / 2 * (GATED ? second : 32);
  }
  __device__ __forceinline__ void load_codes(u32x4 (&c)[NJ], const Walk& w) const {
    const __amdgpu_buffer_rsrc_t rw =
        uniform_buffer(codes + (int64_t)w.s.e * codes_bytes, w.s.rows > 0 ? codes_bytes : 0);
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint32_t r = (uint32_t)(first_column(w, j) + i / 4 * 8 + i % 4);
      c[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rw, (r >> 4) * codes_stride + w.block * 1024 + ((r & 15) | g << 4) * 16, 0, 0);
    }
  }
  // (E2M1: of the lane's weight rows; INT4: of its results.)
  __device__ __forceinline__ void load_scales(decltype(Packed::scales)& v, const Walk& w) const {
    const __amdgpu_buffer_rsrc_t rs =
        uniform_buffer(scales + (int64_t)w.s.e * scales_bytes, w.s.rows > 0 ? scales_bytes : 0);
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (E2M1) {
        const uint32_t r = (uint32_t)(first_column(w, j) + i / 4 * 8 + i % 4);
        v[j] = __builtin_amdgcn_raw_buffer_load_b32(
            rs, (r >> 4) * scales_stride + (w.block * 16 + (r & 15)) * 4, 0, 0);
      } else {
        const uint32_t c = (uint32_t)(first_column(w, j) + g * 8);
        v[j].load(rs,
                  (c >> 4) * scales_stride + w.block * (kGroups * 32) + (c & 15) * Int4Scales<G>::kRow, 0);
      }
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

  // Products with -24 of the wave's quarter of the rows of x at `from`, to `to`.
  __device__ __forceinline__ void products_less(const char* __restrict__ from,
                                                char* __restrict__ to) const {
    static_assert(E2M1 || MI == kNW);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            offset,
            *reinterpret_cast<const bf16x8*>(from + wave * 4096 + from_[q * kSteps + s]), t, 0, 0, 0);
      if (lane < 16) *reinterpret_cast<f32x4*>(to + (q * BM + wave * 16 + lane) * 16) = t;
    }
  }

  // Products of a block with x at `from`, the loads of x kAhead blocks on (wx), to another stage, which
  // saying so (restrict) keeps these reads from waiting for, and those of the next block's codes and
  // scales (wp), which take the place of this block's: the scales when all are used, which saves
  // registers.  rows: rows of the tile that there are (SKIP: products of 16 rows that are all absent
  // are left out).
  __device__ __forceinline__ void multiply(const Walk& wx, const Walk& wp, char* __restrict__ to,
                                           const char* __restrict__ from, const char* __restrict__ less,
                                           int rows, Packed& p) {
    u32x4 then[NJ];
    load_codes(then, wp);
    load_x(wx, to);
    auto fragment = [&](int i, int s) {
      return *reinterpret_cast<const bf16x8*>(from + i * 4096 + from_[s]);
    };
    if constexpr (E2M1) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 b[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          b[j] = decode_e2m1(p.codes[j][s], e2m1_scale((p.scales[j] >> (8 * s)) & 0xffu));
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if (SKIP && i > 0 && rows <= i * 16) break;
          const bf16x8 a = fragment(i, s);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a, acc[i][j], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        bf16x8 b[kSteps][NJ];
        float scale[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s) b[s][j] = decode_int4(p.codes[j][q * kSteps + s]);
#pragma unroll
          for (int r = 0; r < 4; ++r) scale[j][r] = p.scales[j].get(r, q);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if (SKIP && i > 0 && rows <= i * 16) break;
          const f32x4 start =
              *reinterpret_cast<const f32x4*>(less + (q * BM + i * 16 + (lane & 15)) * 16);
          f32x4 part[NJ];
          bf16x8 a[kSteps];
#pragma unroll
          for (int s = 0; s < kSteps; ++s) a[s] = fragment(i, q * kSteps + s);
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[s][j], a[s], s == 0 ? start : part[j],
                                                                0, 0, 0);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[i][j][r] = __builtin_fmaf(scale[j][r], part[j][r], acc[i][j][r]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_scales(p.scales, wp);
#pragma unroll
    for (int j = 0; j < NJ; ++j) p.codes[j] = then[j];
  }

  // acc = x w^T of a tile of `rows` rows.  now: codes and scales of its first block, and of the next
  // tile's afterwards.  advance(walk) goes to the block after: wp is that of the codes that are
  // loaded next, a block ahead, and wx that of x, kAhead ahead.
  template <typename Advance>
  __device__ __forceinline__ void run(char* lds, Walk& wx, Walk& wp, const Advance& advance, int rows,
                                      Packed& now) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int n = 0; n < blocks; ++n) {
      // A tile's first kAhead blocks of x had landed before the last epilogue.  After a later one's
      // loads came scales, and those of a whole block where more are under way than are needed now:
      // this block, and with INT4 the next.
      if (n + (E2M1 ? 0 : 1) < kAhead)
        wait_and_meet<-1>();
      else
        wait_and_meet<kAhead == 1 ? NJ : NJ + QA + 2 * NJ>();
      const int next = stage_after(put), other = 2 * kStages * kStage + kLess - less;
      const int free = put == 0 ? (kStages - 1) * kStage : put - kStage;
      if constexpr (!E2M1) products_less(lds + next, lds + other);
      multiply(wx, wp, lds + free, lds + put, lds + less, rows, now);
      put = next;
      less = other;
      advance(wx);
      advance(wp);
    }
    // The next tile's first blocks have landed before the epilogue's stores are issued.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
};

// The epilogue of a tile: bias, activation, residual, and y.
template <typename P>
__device__ __forceinline__ void tile4_epilogue(const P& p, const ExpertDims& x, const Segment& s,
                                               int col0, const float* bias, const uint16_t* residual,
                                               uint16_t* y) {
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
        const f32x4* q =
            reinterpret_cast<const f32x4*>(bias + (int64_t)s.e * x.Z + col + (P::GATED ? h * x.N : 0));
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
  if constexpr (P::MI > 4) rows_epilogue<P, 4>(p, x, s, c0, bz, residual, y, nullptr);
}

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
  typename P::Walk w{(int)blockIdx.x, {0, 0, 0}, 0, 0};
  auto enter = [&](typename P::Walk& w) {  // the next tile
    w.s.rows = w.block = 0;
    for (; w.number < numbers; w.number += gridDim.x) {
      const Tile t = grid.at(w.number);
      if (!t.live) continue;
      w.s = segment_of<P::BM>(table, off, x.E, t.m);
      w.n0 = t.n * kCols;
      w.number += gridDim.x;
      break;
    }
  };
  auto advance = [&](typename P::Walk& w) {
    if (++w.block >= w4.blocks) enter(w);
  };
  enter(w);
  if (w.s.rows <= 0) return;
  P p(x, w4, a, codes, scales);
  typename P::Walk wx = w, wp = w;
  typename P::Packed packed;
  p.load_codes(packed.codes, wp);
  p.load_scales(packed.scales, wp);
  advance(wp);
  for (int n = 0; n < P::kAhead; ++n) {
    p.load_x(wx, lds + n * P::kStage);
    advance(wx);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (P::kLess > 0) {
    P::template wait_and_meet<-1>();
    p.products_less(lds, lds + p.less);
  }
  while (w.s.rows > 0) {
    p.run(lds, wx, wp, advance, w.s.rows, packed);
    tile4_epilogue(p, x, w.s, w.n0, bias, residual, y);
    enter(w);
  }
}

// The kernel for few rows is taken up to 6 rows an expert on average, up to 80 where the tiles would
// leave half of the CUs without one, and always with INT4 in groups of 32 (Tile4).  Its passes take
// 16 rows where no expert has more or they have up to 12 on average, else 32.  (All by the average, which
// the host has; measured with uniform routing.)  In us, passes of 16, of
// 32, and tiles of 64 rows, INT4 in groups of 128 (E2M1): 64 experts, top-8, 2048 -> 2 x 1024: 8 tokens
// 22, 30, 28 (20, 24, 27), 48 tokens 28, 36, 31 (27, 33, 30), 64 tokens 33, 38, 30 (31, 32, 29), 256
// tokens 69, 67, 40 (67, 55, 37); 30 experts, top-2, 4096 -> 4096: 32 tokens 48, 63, 52 (46, 55, 50), 64
// tokens 56, 70, 55 (55, 61, 53); 8 experts of those, with 128 tiles: 64 tokens 34, 25, 41 (31, 23, 38),
// 256 tokens 82, 64, 74 (73, 55, 63), 512 tokens 139, 106, 75 (122, 90, 65).
bool few4(const ExpertDims& x, const Weights4& w4) {
  const int tiles = ceil_div(x.N, gated(x.act) ? 128 : 256);
  return (!w4.e2m1 && w4.group == 32) || (int64_t)x.rows <= (int64_t)x.E * 6 ||
         ((int64_t)x.rows <= (int64_t)x.E * 80 && (int64_t)x.E * tiles <= kCus / 2);
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
        // Fewer rows at a time where the contraction is too long for 16 and no expert can have more (top-8
        // of 256, 7168 -> 2 x 1024, INT4 in groups of 128: 4 tokens take 46 us in passes of 4, 48 of 16).
        // Not where the average alone is small, since an expert's passes follow one another: 16 tokens
        // take 150 and 148 us, but 162 and 67 under Zipf 1.2, whose busiest expert has 16 rows; 500 tokens,
        // top-1 of 1024, 7168 -> 128: 43 and 44, 1178 and 467 under Zipf; at worst, 16 tokens, top-1 of 128,
        // 7168 -> 2048: 26 and 29, 47 and 27 under Zipf.
        while (cut.rows > 4 && cut.rows * w4.blocks * 256 > F::kXBytes && cut.rows / 2 >= x.T)
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
    if (few4(x, w4)) {
      if (x.T <= 16 || (int64_t)x.rows <= (int64_t)x.E * 12) return few(std::integral_constant<int, 1>());
      return few(std::integral_constant<int, 2>());
    }
    const bool whole = (int64_t)x.rows >= (int64_t)x.E * 96;  // most tiles have all of their rows
    if constexpr (E2M1) {
      if (whole && (int64_t)x.rows * ceil_div(x.N, gated(x.act) ? 128 : 256) >= 128 * 4 * kCus)
        return gated(x.act) ? tiles(Type<Tile4<G, E2M1, true, 8, false>>())
                            : tiles(Type<Tile4<G, E2M1, false, 8, false>>());
    } else if constexpr (G == 128) {
      if (whole)
        return gated(x.act) ? tiles(Type<Tile4<G, E2M1, true, 4, false>>())
                            : tiles(Type<Tile4<G, E2M1, false, 4, false>>());
    }
    if constexpr (E2M1 || G > 32)
      return gated(x.act) ? tiles(Type<Tile4<G, E2M1, true, 4, true>>())
                          : tiles(Type<Tile4<G, E2M1, false, 4, true>>());
    else
      return hipErrorInvalidValue;  // (few4 takes them all)
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
