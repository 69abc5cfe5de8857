// Gradients of the shuffle on gfx950: of the dispatch (a token's row is the
// sum of its receive rows' gradients) and of the combine (a receive row's
// gradient is its token's, weighted; a weight's is a dot product of rows).
//
// Both are bound by HBM: every row is read once and written once.  Like the
// forward movement, the unit of work is a wave that owns one 64-chunk segment
// (512 elements) of a token row, 16 bytes a lane, and finds its receive rows
// in slot_of; a token's segments are spread over the waves of a block where
// the dot products need the whole row.
#include <algorithm>
#include <type_traits>

#include "layer_internal.h"
#include "move_body.h"

namespace moe {
namespace {

template <bool F32>
__device__ __forceinline__ void load_values(const void* p, int64_t chunk, float (&f)[8]) {
  if constexpr (F32) {
    const f32x4* q = static_cast<const f32x4*>(p) + chunk * 2;
    const f32x4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  } else {
    unpack_bf16(load_chunk(static_cast<const u32x4*>(p) + chunk), f);
  }
}

__device__ __forceinline__ u32x4 pack_bf16(const float (&f)[8]) {
  u32x4 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r[q] = bf16_rne(f[2 * q]) | (bf16_rne(f[2 * q + 1]) << 16);
  return r;
}

constexpr int kDispatchGradWaves = 2;

// grad_x[t] = sum over the slots j of grad_recv[row of (t, j)], in float32 in the
// order of the slots.  All rows of a segment are loaded before the first is
// added, so k * 1 KiB are under way a wave.  32768 tokens of 2048 bf16, top-6 (940
// MB): 152 us, 6.2 TB/s; 4096 of 2048 float32, top-8 (168 MB): 25.6 us; 128 of 256, top-2:
// 2.5 us, a launch.
// Wave-items [base, limit) of the batch (one launch of at most kMaxLaunchItems).
template <int KMAX, bool F32>
__global__ __launch_bounds__(kDispatchGradWaves * kWave) void dispatch_grad_kernel(
    Dims d, const u32x4* __restrict__ grad_recv, const int32_t* __restrict__ slot_of,
    void* __restrict__ grad_x, int base, int limit) {
  const uint32_t rows = (uint32_t)(d.T * d.k);
  const Item it = wave_item<1, kDispatchGradWaves>(d, blockIdx.x, base, limit, 0);
  const int64_t at = (int64_t)it.t * d.k;
  int slot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) slot[j] = slot_of[slot_index(at, j, d.k)];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (!(it.live && j < d.k && (uint32_t)slot[j] < rows)) slot[j] = -1;
  u32x4 v[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (slot[j] >= 0 && it.ok) v[j] = load_chunk(&grad_recv[(int64_t)slot[j] * d.chunks + it.c]);
  if (!it.ok) return;
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (slot[j] < 0) continue;
    float f[8];
    unpack_bf16(v[j], f);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += f[q];
  }
  const int64_t i = (int64_t)it.t * d.chunks + it.c;
  if constexpr (F32) {
    f32x4* o = static_cast<f32x4*>(grad_x) + i * 2;
    const f32x4 a = {acc[0], acc[1], acc[2], acc[3]}, b = {acc[4], acc[5], acc[6], acc[7]};
    store_chunk(o, a);
    store_chunk(o + 1, b);
  } else {
    store_chunk(static_cast<u32x4*>(grad_x) + i, pack_bf16(acc));
  }
}

constexpr int kCombineGradWaves = 4;
constexpr int kCombineGradBlocks = 1 << 20;  // tokens a launch at most; more go in further rounds

// One block per token: its waves share the row's segments; each lane keeps
// the k partial dot products of its chunks, which are added over the lanes
// and then over the waves in a fixed order.
//   grad_y[row of (t, j)] = wts[t, j] * grad_out[t]
//   grad_w[t, j] = sum over the columns of grad_out[t] * y[row of (t, j)]
// grad_out is read once for both.  4096 tokens of 2048 float32, top-8 (302 MB): 61 us,
// 5.0 TB/s; 16384 of 7168, top-8 (4.0 GB): 798 us, 5.0 TB/s.  Rows of fewer than 2048
// columns leave waves of their block idle: 16384 tokens of 64, top-8 (36 MB) 78 us, of 256 (143
// MB) 81, bound by their blocks.  Other numbers of waves a
// token, and plain instead of streaming loads and stores, measured equal or worse.
template <int KMAX, bool F32>
__global__ __launch_bounds__(kCombineGradWaves * kWave) void combine_grad_kernel(
    Dims d, const void* __restrict__ grad_out, const u32x4* __restrict__ y,
    const float* __restrict__ wts, const int32_t* __restrict__ slot_of,
    u32x4* __restrict__ grad_y, float* __restrict__ grad_w) {
  __shared__ float s_dot[kCombineGradWaves][KMAX];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const uint32_t rows = (uint32_t)(d.T * d.k);
  for (int64_t t = blockIdx.x; t < d.T; t += gridDim.x) {
    const int64_t at = t * d.k;
    int slot[KMAX];
    float wj[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const int64_t a = slot_index(at, j, d.k);
      slot[j] = slot_of[a];
      wj[j] = wts[a];
      dot[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (!(j < d.k && (uint32_t)slot[j] < rows)) slot[j] = -1;
    for (int c = wave * kWave + lane; c < d.chunks; c += kCombineGradWaves * kWave) {
      u32x4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (slot[j] >= 0) v[j] = load_chunk(&y[(int64_t)slot[j] * d.chunks + c]);
      float g[8];
      load_values<F32>(grad_out, t * d.chunks + c, g);
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (slot[j] < 0) continue;
        float f[8], o[8];
        unpack_bf16(v[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          dot[j] = __builtin_fmaf(g[q], f[q], dot[j]);
          o[q] = wj[j] * g[q];
        }
        store_chunk(&grad_y[(int64_t)slot[j] * d.chunks + c], pack_bf16(o));
      }
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
      if (lane == 0) s_dot[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < d.k) {
      float sum = 0.0f;
      for (int q = 0; q < kCombineGradWaves; ++q) sum += s_dot[q][threadIdx.x];
      grad_w[at + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

template <typename F>
hipError_t by_slots(int k, F f) {
  if (k <= 2) return f(std::integral_constant<int, 2>());
  if (k <= 4) return f(std::integral_constant<int, 4>());
  if (k <= 8) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_dispatch_grad(const Dims& d, const uint16_t* grad_recv, void* grad_x, bool f32,
                                const Work& w, hipStream_t s) {
  const u32x4* gv = reinterpret_cast<const u32x4*>(grad_recv);
  const int64_t items = (int64_t)d.T * d.segs;
  return by_slots(d.k, [&](auto v) {
    constexpr int K = decltype(v)::value;
    hipError_t e = hipSuccess;
    for (int64_t b = 0; b < items && e == hipSuccess; b += kMaxLaunchItems) {
      const int64_t l = std::min(items, b + kMaxLaunchItems);
      e = launch(MOE_KERNEL_DISPATCH_GRAD,
                 f32 ? dispatch_grad_kernel<K, true> : dispatch_grad_kernel<K, false>,
                 dim3((uint32_t)((l - b + kDispatchGradWaves - 1) / kDispatchGradWaves)),
                 dim3(kDispatchGradWaves * kWave), 0, s, d, gv, w.slot_of, grad_x, (int)b, (int)l);
    }
    return e;
  });
}

hipError_t launch_combine_grad(const Dims& d, const void* grad_out, bool f32, const uint16_t* y,
                               const float* wts, uint16_t* grad_y, float* grad_w, const Work& w,
                               hipStream_t s) {
  const u32x4* yv = reinterpret_cast<const u32x4*>(y);
  u32x4* gv = reinterpret_cast<u32x4*>(grad_y);
  return by_slots(d.k, [&](auto v) {
    constexpr int K = decltype(v)::value;
    return launch(MOE_KERNEL_COMBINE_GRAD,
                  f32 ? combine_grad_kernel<K, true> : combine_grad_kernel<K, false>,
                  dim3((uint32_t)std::min(d.T, kCombineGradBlocks)),
                  dim3(kCombineGradWaves * kWave), 0, s, d, grad_out, yv, wts, w.slot_of, gv,
                  grad_w);
  });
}

}  // namespace moe
