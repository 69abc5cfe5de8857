// Layer norm and RMS norm of the residual stream's rows on gfx950, after the
// residual addition, and their gradient.
//   total = x + residual (rounded to x's type), h = (total - mean) rstd, y = h gamma + beta
//   g = grad_y gamma, grad_x = rstd (g - mean(g) - h mean(g h)) + grad_total (RMS: no mean(g)),
//   grad_gamma = sum of grad_y h over the rows, grad_beta = sum of grad_y
//
// Both are bound by HBM: a row is read once and kept in registers between the
// statistics and the result (the variance from the differences to the mean, not from the squares'
// sum, which would cancel).  A row belongs to W waves (or to 16 or 32 lanes of one, where it is
// narrow), 8 columns a lane and chunk; the statistics are folded over the lanes by
// data-parallel moves and over the waves through LDS, in a fixed order.  Blocks
// stay and take row after row, so that the weights are read once a block, and
// a row's loads are under way while the row before it is reduced.  Everything between load and store
// is float32; the total is rounded before the statistics are taken, so that the gradient, which
// reads it back, has the same ones.
//
// Measured: forward, 32768 x 2048 with residual and total, float32 to bf16: 178 us, 5.3 TB/s (with
// streaming loads 200, with streaming stores 183); 16 x 7168: 4.1 us, a launch and a row's chain of
// load, fold and store; 16384 x 16384 bf16: 404 us, 5.3 TB/s.  Gradient, 16384 x 7168 bf16 with all
// outputs: 176 us, 5.3 TB/s; 16384 x 16384: 469 us, 4.6 TB/s; 4099 x 1000: 16.5 us with the sums' launch.
#include <algorithm>
#include <type_traits>

#include "block_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kCus = 256;
constexpr int kMaxWaves = 16;

// How the rows are spread: `waves` waves a row (1 where lanes < 64), `rows` rows a block at a time.
struct Spread {
  int32_t chunks;  // of 8 columns
  int32_t waves, rows;
};

// Eight values of a row, as memory holds them.
template <bool F32>
struct Raw;
template <>
struct Raw<false> {
  u32x4 v;
};
template <>
struct Raw<true> {
  f32x4 lo, hi;
};

__device__ __forceinline__ void load(const void* p, int64_t chunk, Raw<false>& r) {
  r.v = static_cast<const u32x4*>(p)[chunk];
}
__device__ __forceinline__ void load(const void* p, int64_t chunk, Raw<true>& r) {
  const f32x4* q = static_cast<const f32x4*>(p) + chunk * 2;
  r.lo = q[0];
  r.hi = q[1];
}

__device__ __forceinline__ void values(const Raw<false>& r, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(r.v[q] << 16);
    f[2 * q + 1] = __uint_as_float(r.v[q] & 0xffff0000u);
  }
}
__device__ __forceinline__ void values(const Raw<true>& r, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[q] = r.lo[q];
    f[4 + q] = r.hi[q];
  }
}

// Rounded to the type (nearest even).
template <bool F32>
__device__ __forceinline__ Raw<F32> rounded(const float (&f)[8]) {
  Raw<F32> r;
  if constexpr (F32) {
    r.lo = f32x4{f[0], f[1], f[2], f[3]};
    r.hi = f32x4{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r.v[q] = __builtin_bit_cast(
          uint32_t, __builtin_convertvector(f32x2{f[2 * q], f[2 * q + 1]}, bf16x2));
  }
  return r;
}

__device__ __forceinline__ void store(void* p, int64_t chunk, const Raw<false>& r) {
  static_cast<u32x4*>(p)[chunk] = r.v;
}
__device__ __forceinline__ void store(void* p, int64_t chunk, const Raw<true>& r) {
  f32x4* q = static_cast<f32x4*>(p) + chunk * 2;
  q[0] = r.lo;
  q[1] = r.hi;
}

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// v added over the other row of 16 lanes (of each pair), and over the other half of the wave.
__device__ __forceinline__ float add_across_16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_across_32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over each L consecutive lanes, in every one of them.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  constexpr int kRor = 0x120;  // rotations in a row of 16
  v += moved<kRor + 8>(v);
  v += moved<kRor + 4>(v);
  v += moved<kRor + 2>(v);
  v += moved<kRor + 1>(v);
  if constexpr (L >= 32) v = add_across_16(v);
  if constexpr (L >= 64) v = add_across_32(v);
  return v;
}

// A lane's place: the row of its block that it works on, and its chunks of it.
template <int L, int CH>
struct Place {
  int row;              // of the block's `rows`
  int first_wave;       // of the row's waves
  int chunk[CH];
  bool live[CH];
  __device__ __forceinline__ explicit Place(const Spread& s) {
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    static_assert(L == kWave || CH == 1);
    if constexpr (L == kWave) {
      row = wave / s.waves;
      first_wave = row * s.waves;
    } else {
      row = wave * (kWave / L) + lane / L;
      first_wave = wave;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      chunk[i] = L == kWave ? (i * s.waves + wave - first_wave) * kWave + lane : lane % L;
      live[i] = chunk[i] < s.chunks;
    }
  }
};

// Sum over the row's lanes, in every one of them; slot: kMaxWaves values in LDS that no wave
// reads any more.  Meets the block's other waves where a row has several.
template <int L>
__device__ __forceinline__ float row_sum(float v, const Spread& s, int first_wave, float* slot) {
  v = lane_sum<L>(v);
  if (L < kWave || s.waves == 1) return v;
  slot[threadIdx.x / kWave] = v;  // the same value from every lane
  __syncthreads();
  float t = 0.0f;
  for (int q = 0; q < s.waves; ++q) t += slot[first_wave + q];
  return t;
}

// eight weights of a column chunk (`none` where there are no weights)
__device__ __forceinline__ void weights(const float* p, int chunk, bool live, float none,
                                        float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = none;
  if (p == nullptr || !live) return;
  Raw<true> r;
  load(p, chunk, r);
  values(r, f);
}

template <bool XF32, bool YF32, int L, int CH>
__global__ __launch_bounds__(kMaxWaves * kWave) void norm_kernel(
    NormDims n, Spread s, const void* __restrict__ x, const void* __restrict__ residual,
    const float* __restrict__ gamma, const float* __restrict__ beta, void* __restrict__ y,
    void* __restrict__ total, float* __restrict__ stats) {
  __shared__ float slots[2][kMaxWaves];
  const Place<L, CH> at(s);
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    weights(gamma, at.chunk[i], at.live[i], 1.0f, w[i]);
    weights(beta, at.chunk[i], at.live[i], 0.0f, b[i]);
  }
  const float share = 1.0f / (float)n.H;
  Raw<XF32> vx[CH], vr[CH];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (row >= n.T || !at.live[i]) continue;
      load(x, row * s.chunks + at.chunk[i], vx[i]);
      if (residual != nullptr) load(residual, row * s.chunks + at.chunk[i], vr[i]);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * s.rows;
  int64_t base = (int64_t)blockIdx.x * s.rows;
  int turn = 0;
  fetch(base + at.row);
  for (; base < n.T; base += stride, turn ^= 1) {  // the same number of turns for every wave
    const int64_t row = base + at.row;
    const bool in = row < n.T;
    float f[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!in || !at.live[i]) {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[i][q] = 0.0f;
        continue;
      }
      values(vx[i], f[i]);
      if (residual != nullptr) {
        float r[8];
        values(vr[i], r);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[i][q] += r[q];
        const Raw<XF32> t = rounded<XF32>(f[i]);
        values(t, f[i]);
        if (total != nullptr) store(total, row * s.chunks + at.chunk[i], t);
      }
    }
    fetch(row + stride);
    float mean = 0.0f;
    if (!n.rms) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) sum += f[i][q];
      mean = row_sum<L>(sum, s, at.first_wave, slots[0]) * share;
    }
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] -= mean;
        if (at.live[i]) squares = __builtin_fmaf(f[i][q], f[i][q], squares);
      }
    // The two barriers of a turn keep a wave from writing slots that another still reads; the RMS
    // norm has one, and takes the slots in turn.
    squares = row_sum<L>(squares, s, at.first_wave, slots[n.rms ? turn : 1]);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(squares, share, n.eps));
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!at.live[i]) continue;
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = __builtin_fmaf(f[i][q] * rstd, w[i][q], b[i][q]);
      store(y, row * s.chunks + at.chunk[i], rounded<YF32>(o));
    }
    if (stats != nullptr && at.chunk[0] == 0)
      reinterpret_cast<f32x2*>(stats)[row] = f32x2{mean, rstd};
  }
}

// Gradient: of the rows, and a block's sums of the weights' gradients (rows blockIdx.x of the
// partial sums, or the sums themselves where there is one block).  A lane adds up its columns over the
// block's rows in registers, the block's rows at a time are joined once at the end (in one pass over
// LDS), and the blocks' sums by norm_sum_kernel, in a fixed order and with no atomics: 256 rows of
// partial sums cost 2% of the traffic of 16384 rows.
template <bool XF32, bool YF32, int L, int CH>
__global__ __launch_bounds__(kMaxWaves * kWave) void norm_grad_kernel(
    NormDims n, Spread s, const void* __restrict__ gy, const void* __restrict__ x,
    const float* __restrict__ stats, const float* __restrict__ gamma,
    const void* __restrict__ gtotal, void* __restrict__ gx, float* __restrict__ ggamma,
    float* __restrict__ gbeta) {
  __shared__ float slots[2][2][kMaxWaves];
  extern __shared__ float sums[];  // [parts][H] where a block's sums come in several parts: 32 KiB at most
  const Place<L, CH> at(s);
  float w[CH][8], sg[CH][8], sb[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    weights(gamma, at.chunk[i], at.live[i], 1.0f, w[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) sg[i][q] = sb[i][q] = 0.0f;
  }
  // With two chunks a lane there are no registers for the loads of a row ahead, and gtotal is
  // loaded where it is added.  (Even so 40 to 56 bytes a lane are in scratch: 128 registers, of which
  // weights and sums keep 48.)
  constexpr bool kAhead = CH == 1;
  const bool joined = gtotal != nullptr && gx != nullptr;
  const float share = 1.0f / (float)n.H;
  Raw<XF32> vx[CH], vt[CH];
  Raw<YF32> vg[CH];
  f32x2 stat = {0.0f, 0.0f};
  auto fetch = [&](int64_t row) {
    if (row >= n.T) return;
    stat = reinterpret_cast<const f32x2*>(stats)[row];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!at.live[i]) continue;
      load(x, row * s.chunks + at.chunk[i], vx[i]);
      load(gy, row * s.chunks + at.chunk[i], vg[i]);
      if (kAhead && joined) load(gtotal, row * s.chunks + at.chunk[i], vt[i]);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * s.rows;
  int64_t base = (int64_t)blockIdx.x * s.rows;
  int turn = 0;
  if (kAhead) fetch(base + at.row);
  for (; base < n.T; base += stride, turn ^= 1) {  // the same number of turns for every wave
    const int64_t row = base + at.row;
    const bool in = row < n.T;
    if (!kAhead) fetch(row);
    const float mean = stat[0], rstd = stat[1];
    float h[CH][8], g[CH][8], along = 0.0f, sum = 0.0f;
    Raw<XF32> now[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const bool on = in && at.live[i];
      if (on) {
        values(vx[i], h[i]);
        values(vg[i], g[i]);
        now[i] = vt[i];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        h[i][q] = on ? (h[i][q] - mean) * rstd : 0.0f;
        g[i][q] = on ? g[i][q] : 0.0f;
        sg[i][q] = __builtin_fmaf(g[i][q], h[i][q], sg[i][q]);
        sb[i][q] += g[i][q];
        g[i][q] *= w[i][q];
        along = __builtin_fmaf(g[i][q], h[i][q], along);
        sum += g[i][q];
      }
    }
    if (kAhead) fetch(row + stride);
    if (gx == nullptr) continue;
    along = lane_sum<L>(along);
    if (!n.rms) sum = lane_sum<L>(sum);
    if (L == kWave && s.waves > 1) {
      // Two buffers in turn: a wave that is a turn ahead has met the others after their reads of
      // the turn before.
      float (&slot)[2][kMaxWaves] = slots[turn];
      slot[0][threadIdx.x / kWave] = along;
      slot[1][threadIdx.x / kWave] = sum;
      __syncthreads();
      along = sum = 0.0f;
      for (int q = 0; q < s.waves; ++q) {
        along += slot[0][at.first_wave + q];
        sum += slot[1][at.first_wave + q];
      }
    }
    if (!in) continue;
    along *= share;
    sum = n.rms ? 0.0f : sum * share;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!at.live[i]) continue;
      float o[8], t[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = rstd * __builtin_fmaf(-h[i][q], along, g[i][q] - sum);
      if (joined) {
        if (!kAhead) load(gtotal, row * s.chunks + at.chunk[i], now[i]);
        values(now[i], t);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += t[q];
      }
      store(gx, row * s.chunks + at.chunk[i], rounded<XF32>(o));
    }
  }

  // The block's sums: over the rows of a wave, then over the block's rows in order.
  auto put = [&](float* out, float (&v)[CH][8]) {
    if (out == nullptr) return;
    float* to = out + (int64_t)blockIdx.x * n.H;
    if constexpr (L < kWave) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if constexpr (L < 32) v[0][q] = add_across_16(v[0][q]);
        v[0][q] = add_across_32(v[0][q]);
      }
    }
    const int parts = L < kWave ? blockDim.x / kWave : s.rows;
    const int part = L < kWave ? at.first_wave : at.row;
    const bool mine = L == kWave || threadIdx.x % kWave < L;
    float* own = parts == 1 ? to : sums + part * n.H;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (mine && at.live[i]) store(own, at.chunk[i], rounded<true>(v[i]));
    if (parts == 1) return;
    __syncthreads();
    for (int c = threadIdx.x * 4; c < n.H; c += blockDim.x * 4) {
      f32x4 t = *reinterpret_cast<const f32x4*>(sums + c);
      for (int p = 1; p < parts; ++p) t += *reinterpret_cast<const f32x4*>(sums + p * n.H + c);
      *reinterpret_cast<f32x4*>(to + c) = t;
    }
    __syncthreads();
  };
  put(ggamma, sg);
  put(gbeta, sb);
}

// Column sums of the partial rows: 64 columns a block, 16 lanes of four columns, each of 16
// parts adds every 16th row in order, then the parts are added in order.
constexpr int kSumParts = 16;
__global__ __launch_bounds__(256) void norm_sum_kernel(const float* __restrict__ partial, int rows,
                                                       int H, float* __restrict__ ggamma,
                                                       float* __restrict__ gbeta) {
  __shared__ f32x4 part[kSumParts][16];
  float* out = blockIdx.y == 0 ? ggamma : gbeta;
  if (out == nullptr) return;
  const float* from = partial + (int64_t)blockIdx.y * rows * H;
  const int lane = threadIdx.x % 16, p = threadIdx.x / 16;
  const int col = (blockIdx.x * 16 + lane) * 4;
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < H) {
#pragma unroll 4
    for (int r = p; r < rows; r += kSumParts)
      t += *reinterpret_cast<const f32x4*>(from + (int64_t)r * H + col);
  }
  part[p][lane] = t;
  __syncthreads();
  if (p != 0 || col >= H) return;
#pragma unroll
  for (int q = 1; q < kSumParts; ++q) t += part[q][lane];
  *reinterpret_cast<f32x4*>(out + col) = t;
}

// Lanes a row where it is narrower than a wave's 64 chunks.
int lanes_of(int chunks) { return chunks <= 16 ? 16 : chunks <= 32 ? 32 : kWave; }

// Chunks a lane: one while 16 waves cover the row.
int chunks_of(int chunks) { return chunks <= kMaxWaves * kWave ? 1 : 2; }
static_assert(kNormMaxColumns == 2 * kMaxWaves * kWave * 8);

// A block of at most `most` waves (as many as a row needs, if that is more).
Spread spread(const NormDims& n, int most, int* threads) {
  const int chunks = n.H / 8, lanes = lanes_of(chunks), ch = chunks_of(chunks);
  const int waves = (chunks + ch * kWave - 1) / (ch * kWave);
  const int rows = std::max(most / waves, 1);
  *threads = rows * waves * kWave;
  return Spread{chunks, waves, rows * (kWave / lanes)};
}

constexpr int kForwardWaves = 4;

template <int V>
using Int = std::integral_constant<int, V>;

template <typename F>
hipError_t with_widths(int chunks, F f) {
  const int lanes = lanes_of(chunks), ch = chunks_of(chunks);
  if (lanes == 16) return f(Int<16>(), Int<1>());
  if (lanes == 32) return f(Int<32>(), Int<1>());
  if (ch == 1) return f(Int<64>(), Int<1>());
  return f(Int<64>(), Int<2>());
}

template <typename F>
hipError_t with_types(const NormDims& n, F f) {
  if (n.x_f32) return n.y_f32 ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
  return n.y_f32 ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}

}  // namespace

// Up to four turns of one block, a block does it all: 128 x 256 takes 9.0 us so and 7.8 with two launches
// in a captured graph, 10.2 and 14.3 from a program, whose launches cost more than the turns.
int norm_partials(const NormDims& n) {
  int threads;
  const Spread s = spread(n, kMaxWaves, &threads);
  const int turns = (n.T + s.rows - 1) / s.rows;
  return turns <= 4 ? 1 : std::min(turns, kCus);
}

hipError_t launch_norm(const NormDims& n, const void* x, const void* residual, const float* gamma,
                       const float* beta, void* y, void* total, float* stats, hipStream_t s) {
  int threads;
  const Spread sp = spread(n, kForwardWaves, &threads);
  const int blocks = std::min((n.T + sp.rows - 1) / sp.rows, kCus * std::max(2048 / threads, 1));
  return with_types(n, [&](auto xf, auto yf) {
    return with_widths(sp.chunks, [&](auto l, auto c) {
      return launch(MOE_KERNEL_NORM, norm_kernel<xf(), yf(), l(), c()>, dim3(blocks), dim3(threads), 0,
                    s, n, sp, x, residual, gamma, beta, y, total, stats);
    });
  });
}

hipError_t launch_norm_grad(const NormDims& n, const void* gy, const void* total,
                            const float* stats, const float* gamma, const void* gtotal, void* gx,
                            float* ggamma, float* gbeta, float* partial, hipStream_t s) {
  int threads;
  const Spread sp = spread(n, kMaxWaves, &threads);
  const bool sums = ggamma != nullptr || gbeta != nullptr;
  const int rows = norm_partials(n);
  float* pg = rows > 1 && ggamma ? partial : ggamma;
  float* pb = rows > 1 && gbeta ? partial + (int64_t)rows * n.H : gbeta;
  const int turns = (n.T + sp.rows - 1) / sp.rows;
  const int blocks = sums ? rows : std::min(turns, kCus);
  // A part for each of the block's rows (or waves of several rows) at a time.
  const int parts = threads / (sp.waves * kWave);
  const int lds = sums && parts > 1 ? parts * n.H * (int)sizeof(float) : 0;
  const hipError_t e = with_types(n, [&](auto xf, auto yf) {
    return with_widths(sp.chunks, [&](auto l, auto c) {
      return launch(MOE_KERNEL_NORM_GRAD, norm_grad_kernel<xf(), yf(), l(), c()>, dim3(blocks),
                    dim3(threads), lds, s, n, sp, gy, total, stats, gamma, gtotal, gx,
                    pg, pb);
    });
  });
  if (e != hipSuccess || !sums || rows == 1) return e;
  return launch(MOE_KERNEL_NORM_SUM, norm_sum_kernel, dim3((n.H + 63) / 64, 2), dim3(256), 0, s, partial,
                rows, n.H, ggamma, gbeta);
}

}  // namespace moe
