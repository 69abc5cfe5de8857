// The router on gfx950: the k experts of each token and their combine
// weights from the gate logits, and the gradient of the logits.
//
// One wave per token; lane l holds the logits of experts i * 64 + l, so the
// row is read once, coalesced, and stays in registers.  Choice: every key
// becomes an unsigned number of the same order; k rounds find the largest
// with a wave-wide maximum of data-parallel moves, and the lowest expert that
// holds it with a ballot for each i.
//
// Weights: with p the softmax or the sigmoid, a renormalised weight is
// p_j / sum_i p_i over the selected = exp(l_j - m) / sum_i exp(l_i - m) with
// l the logit (softmax) or log sigmoid(logit) = min(x, 0) - log1p(exp(-|x|))
// and m their maximum, so no logit, however far from 0, under- or overflows it.
#include <algorithm>
#include <type_traits>

#include "layer_internal.h"
#include "moe_device.h"

namespace moe {
namespace {

constexpr int kRouterWaves = 4;
constexpr int kRouterMaxBlocks = 1 << 16;  // tokens beyond are taken in further rounds

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (F32)
    return static_cast<const float*>(p)[i];
  else
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return ((u >> 16) | 0x40u) & 0xffffu;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// A NaN logit counts as -infinity for the weights.
__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -INFINITY; }

// Order-preserving bits of a key: NaN 1, then -infinity ... +infinity; 0 is
// left for an expert that may not be chosen.  -0 counts as 0.
__device__ __forceinline__ uint32_t key_bits(float v) {
  if (v != v) return 1u;
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// v in another lane of the row of 16 (or of the rows before), `other` where
// there is none: data-parallel moves, no LDS.
constexpr int kRowShr = 0x110, kBcast15 = 0x142, kBcast31 = 0x143;
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t moved(uint32_t other, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)other, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float moved(float other, float v) {
  return __uint_as_float(moved<CTRL, ROWS>(__float_as_uint(other), __float_as_uint(v)));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Folds f over the first 16 lanes (into lane 15) or all 64 (into lane 63) and
// gives every lane the result.  The order is fixed.
template <bool WHOLE, typename T, typename F>
__device__ __forceinline__ T fold(T v, T none, F f) {
  v = f(v, moved<kRowShr + 1>(none, v));
  v = f(v, moved<kRowShr + 2>(none, v));
  v = f(v, moved<kRowShr + 4>(none, v));
  v = f(v, moved<kRowShr + 8>(none, v));
  if constexpr (WHOLE) {
    v = f(v, moved<kBcast15, 0xa>(none, v));
    v = f(v, moved<kBcast31, 0xc>(none, v));
  }
  constexpr int last = WHOLE ? kWave - 1 : 15;
  if constexpr (std::is_same_v<T, float>)
    return lane_value(v, last);
  else
    return (T)__builtin_amdgcn_readlane((int)v, last);
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <bool WHOLE>
__device__ __forceinline__ float fold_max(float v) {
  return fold<WHOLE>(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

template <bool WHOLE>
__device__ __forceinline__ float fold_sum(float v) {
  return fold<WHOLE>(v, 0.0f, [](float a, float b) { return a + b; });
}

// The entry with the largest key, the lowest number first: entry i * 64 + lane
// is key[i].  Sets its key to 0 (no entry).
template <int V>
__device__ __forceinline__ int take_largest(uint32_t (&key)[V]) {
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = larger(best, key[i]);
  best = fold<true>(best, 0u, larger);
  int found = -1;
#pragma unroll
  for (int i = V - 1; i >= 0; --i) {
    const uint64_t at = __ballot(key[i] == best);
    found = at != 0 ? i * kWave + __builtin_ctzll(at) : found;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = found == i * kWave + (int)(threadIdx.x % kWave) ? 0u : key[i];
  return found;
}

// exp(x - m) for x <= m, with exp(inf - inf) = 1 (the limit of equal logits)
// and 0 where every logit is -infinity.
__device__ __forceinline__ float exp_below(float x, float m) {
  if (x == -INFINITY) return 0.0f;
  return x == m ? 1.0f : expf(x - m);
}

__device__ __forceinline__ float log_sigmoid(float x) {
  return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Score of the selected logit x that lane j (< k) holds, before the scale;
// lanes without a selected logit pass has = false and get 0.  row_max and
// row_sum: softmax statistics of the whole row (used without renormalising).
__device__ __forceinline__ float selected_score(const moe_router_config& c, float x, bool has,
                                                float row_max, float row_sum) {
  if (c.renormalise) {
    const float l = !has ? -INFINITY : c.score == MOE_SCORE_SIGMOID ? log_sigmoid(x) : x;
    const float m = fold_max<false>(l);
    const float e = exp_below(l, m);
    const float sum = fold_sum<false>(e);
    return sum > 0.0f ? e / sum : 0.0f;
  }
  if (!has) return 0.0f;
  if (c.score == MOE_SCORE_SIGMOID) return sigmoid(x);
  return row_sum > 0.0f ? exp_below(x, row_max) / row_sum : 0.0f;
}

// V: logits per lane, ceil(E / 64).
template <int V, bool F32>
__global__ __launch_bounds__(kRouterWaves * kWave) void router_kernel(
    Dims d, moe_router_config c, const void* __restrict__ logits, const float* __restrict__ bias,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  __shared__ float s_key[kRouterWaves][V * kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave; t < d.T;
       t += (int64_t)gridDim.x * kRouterWaves) {
    float x[V], v[V];
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * kWave + lane;
      x[i] = e < d.E ? load_logit<F32>(logits, t * d.E + e) : -INFINITY;
      v[i] = bias != nullptr && e < d.E ? x[i] + bias[e] : x[i];
      key[i] = e < d.E ? key_bits(v[i]) : 0;
    }
    if (c.nodes_per_token > 0) {
      // The largest two keys of each node: `share` lanes scan a node's
      // consecutive experts and join what they found.  The waves of a block
      // use their own part of s_key and do not wait for each other, only for
      // their own writes.
#pragma unroll
      for (int i = 0; i < V; ++i) s_key[wave][i * kWave + lane] = no_nan(v[i]);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      int share = kWave;
      while (share * d.N > kWave) share >>= 1;
      const int n = lane / share;
      const int r0 = min(n, d.N) * d.G, r1 = min(n + 1, d.N) * d.G;
      const int e0 = r0 * d.ebase + min(r0, d.erem), e1 = r1 * d.ebase + min(r1, d.erem);
      float a = -INFINITY, b = -INFINITY;
      for (int e = e0 + lane % share; e < e1; e += share) {
        const float q = s_key[wave][e];
        b = fmaxf(b, fminf(a, q));
        a = fmaxf(a, q);
      }
      for (int s = share >> 1; s > 0; s >>= 1) {
        const float a2 = __shfl_xor(a, s), b2 = __shfl_xor(b, s);
        b = fmaxf(fmaxf(b, b2), fminf(a, a2));
        a = fmaxf(a, a2);
      }
      // two opposite infinities: the larger one decides
      const float worth = e1 - e0 < 2 || a == INFINITY ? a : a + b;
      uint32_t node[1] = {n < d.N && lane % share == 0 ? key_bits(worth) : 0};
      bool kept[V];
#pragma unroll
      for (int i = 0; i < V; ++i) kept[i] = false;
      for (int m = 0; m < c.nodes_per_token; ++m) {
        const int k0 = take_largest(node) / share * d.G, k1 = k0 + d.G;
        const int f0 = k0 * d.ebase + min(k0, d.erem), f1 = k1 * d.ebase + min(k1, d.erem);
#pragma unroll
        for (int i = 0; i < V; ++i)
          kept[i] = kept[i] || (i * kWave + lane >= f0 && i * kWave + lane < f1);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = kept[i] ? key[i] : 0;
      __builtin_amdgcn_wave_barrier();  // the next token's keys overwrite s_key
    }
    int id = 0;  // lane j (< k): the j-th expert
    for (int j = 0; j < d.k; ++j) {
      const int e = take_largest(key);
      id = lane == j ? e : id;
    }
    const bool has = lane < d.k;
    const float xs = has ? load_logit<F32>(logits, t * d.E + id) : 0.0f;
    float row_max = 0.0f, row_sum = 0.0f;
    if (c.score == MOE_SCORE_SOFTMAX && !c.renormalise) {
      row_max = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, no_nan(x[i]));
      row_max = fold_max<true>(row_max);
#pragma unroll
      for (int i = 0; i < V; ++i) row_sum += exp_below(no_nan(x[i]), row_max);
      row_sum = fold_sum<true>(row_sum);
    }
    const float p = selected_score(c, no_nan(xs), has, row_max, row_sum);
    if (has) {
      topk_idx[t * d.k + lane] = id;
      topk_w[t * d.k + lane] = c.scale * p;
    }
  }
}

// Gradient.  With g_j = scale * grad_w[j] and p_j the selected scores:
//   renormalised: grad_j = p_j (g_j - sum_i p_i g_i) * (1 - sigmoid(x_j) for
//                 the sigmoid, whose log has that slope), 0 elsewhere;
//   softmax:      grad_e = p_e (g_e - sum_i p_i g_i) over all e, g_e = 0 for
//                 the experts that are not selected;
//   sigmoid:      grad_j = g_j p_j (1 - p_j), 0 elsewhere.
template <int V, bool F32>
__global__ __launch_bounds__(kRouterWaves * kWave) void router_grad_kernel(
    Dims d, moe_router_config c, const void* __restrict__ logits,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ grad_w,
    void* __restrict__ grad_logits) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const bool whole = c.score == MOE_SCORE_SOFTMAX && !c.renormalise;
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave; t < d.T;
       t += (int64_t)gridDim.x * kRouterWaves) {
    int id = -1;
    float g = 0.0f;
    if (lane < d.k) {
      id = topk_idx[t * d.k + lane];
      g = c.scale * grad_w[t * d.k + lane];
    }
    const bool has = (uint32_t)id < (uint32_t)d.E;
    const float xs = has ? no_nan(load_logit<F32>(logits, t * d.E + id)) : -INFINITY;
    float p[V];
    float row_max = 0.0f, row_sum = 0.0f;
    if (whole) {
      row_max = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        p[i] = e < d.E ? no_nan(load_logit<F32>(logits, t * d.E + e)) : -INFINITY;
        row_max = fmaxf(row_max, p[i]);
      }
      row_max = fold_max<true>(row_max);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = exp_below(p[i], row_max);
        row_sum += p[i];
      }
      row_sum = fold_sum<true>(row_sum);
      const float inv = row_sum > 0.0f ? 1.0f / row_sum : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    const float ps = selected_score(c, xs, has, row_max, row_sum);
    float gj = 0.0f, dot = 0.0f;  // this lane's entry of the gradient
    if (c.renormalise || whole) dot = fold_sum<false>(has ? ps * g : 0.0f);
    if (c.renormalise) {
      gj = ps * (g - dot);
      if (c.score == MOE_SCORE_SIGMOID) gj *= 1.0f / (1.0f + expf(xs));  // 1 - sigmoid(xs)
    } else if (whole) {
      gj = ps * g;
    } else {
      gj = g * ps * (1.0f / (1.0f + expf(xs)));
    }
    if (!has) gj = 0.0f;
    float out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = whole ? -p[i] * dot : 0.0f;
    for (int j = 0; j < d.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float a = lane_value(gj, j);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e == i * kWave + lane) out[i] += a;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * kWave + lane;
      if (e >= d.E) continue;
      if constexpr (F32)
        static_cast<float*>(grad_logits)[t * d.E + e] = out[i];
      else
        static_cast<uint16_t*>(grad_logits)[t * d.E + e] = (uint16_t)bf16_bits(out[i]);
    }
  }
}

dim3 router_grid(const Dims& d) {
  return dim3((uint32_t)std::min<int64_t>(((int64_t)d.T + kRouterWaves - 1) / kRouterWaves,
                                          kRouterMaxBlocks));
}

// Calls f with ceil(E / 64), rounded up to a power of two, as a constant.
template <typename F>
hipError_t by_experts(int E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 1>());
  if (E <= 128) return f(std::integral_constant<int, 2>());
  if (E <= 256) return f(std::integral_constant<int, 4>());
  if (E <= 512) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_router(const Dims& d, const moe_router_config& c, const void* logits, bool f32,
                         const float* bias, int32_t* topk_idx, float* topk_w, hipStream_t s) {
  return by_experts(d.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    return launch(MOE_KERNEL_ROUTER, f32 ? router_kernel<V, true> : router_kernel<V, false>,
                  router_grid(d), dim3(kRouterWaves * kWave), 0, s, d, c, logits, bias, topk_idx,
                  topk_w);
  });
}

hipError_t launch_router_grad(const Dims& d, const moe_router_config& c, const void* logits,
                              bool f32, const int32_t* topk_idx, const float* grad_w,
                              void* grad_logits, hipStream_t s) {
  return by_experts(d.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    return launch(MOE_KERNEL_ROUTER_GRAD,
                  f32 ? router_grad_kernel<V, true> : router_grad_kernel<V, false>, router_grid(d),
                  dim3(kRouterWaves * kWave), 0, s, d, c, logits, topk_idx, grad_w, grad_logits);
  });
}

}  // namespace moe
