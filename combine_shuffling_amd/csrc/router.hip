// The router on gfx950: the k experts of each token and their combine
// weights from the gate logits, and the gradient of the logits.
//
// One wave per token; lane l holds the logits of experts i * 64 + l, so the
// row is read once, coalesced, and stays in registers.  Choice: every key
// becomes one unsigned 64-bit number, the key's float order above the
// complement of the expert id, so the largest number is the largest key with
// ties to the lower id and no two numbers are equal; k rounds of a wave-wide
// maximum give the ids in descending order.
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

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint64_t o = __shfl_xor(v, s);
    v = o > v ? o : v;
  }
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
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
    const float m = wave_max(l);
    const float e = exp_below(l, m);
    const float sum = wave_sum(e);
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
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave; t < d.T;
       t += (int64_t)gridDim.x * kRouterWaves) {
    float x[V], v[V];
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * kWave + lane;
      x[i] = e < d.E ? load_logit<F32>(logits, t * d.E + e) : -INFINITY;
      v[i] = bias != nullptr && e < d.E ? x[i] + bias[e] : x[i];
      key[i] = e < d.E ? (uint64_t)key_bits(v[i]) << 32 | (uint32_t)~e : 0;
    }
    if (c.nodes_per_token > 0) {
      // Lane n sums node n's two largest keys (its experts are consecutive).
      // The waves of a block use their own part of s_key and do not wait for
      // each other, only for their own writes.
#pragma unroll
      for (int i = 0; i < V; ++i) s_key[wave][i * kWave + lane] = v[i];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      uint64_t node = 0;
      if (lane < d.N) {
        const int r0 = lane * d.G, r1 = r0 + d.G;
        const int e0 = r0 * d.ebase + min(r0, d.erem), e1 = r1 * d.ebase + min(r1, d.erem);
        float a = -INFINITY, b = -INFINITY;
        for (int e = e0; e < e1; ++e) {
          const float q = no_nan(s_key[wave][e]);
          b = fmaxf(b, fminf(a, q));
          a = fmaxf(a, q);
        }
        // two opposite infinities: the larger one decides
        const float worth = e1 - e0 < 2 || a == INFINITY ? a : a + b;
        node = (uint64_t)key_bits(worth) << 32 | (uint32_t)~lane;
      }
      uint64_t kept = 0;  // bit n: node n may be chosen
      for (int m = 0; m < c.nodes_per_token; ++m) {
        const uint64_t best = wave_max(node);
        const int n = (int)~(uint32_t)best;
        kept |= 1ull << (n & 63);
        if (lane == n) node = 0;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        if (e < d.E && !(kept >> (split_part(e, d.ebase, d.erem) / d.G) & 1)) key[i] = 0;
      }
      __builtin_amdgcn_wave_barrier();  // the next token's keys overwrite s_key
    }
    int id = 0;      // lane j (< k): the j-th expert
    float xs = 0.0f;  // and its logit
    for (int j = 0; j < d.k; ++j) {
      uint64_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
      best = wave_max(best);
      const int e = (int)~(uint32_t)best;
      if (lane == j) id = e;
      float mine = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] == best) {
          key[i] = 0;
          mine = x[i];
        }
      const float got = __shfl(mine, e & (kWave - 1));
      if (lane == j) xs = got;
    }
    float row_max = 0.0f, row_sum = 0.0f;
    if (c.score == MOE_SCORE_SOFTMAX && !c.renormalise) {
      row_max = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, no_nan(x[i]));
      row_max = wave_max(row_max);
#pragma unroll
      for (int i = 0; i < V; ++i) row_sum += exp_below(no_nan(x[i]), row_max);
      row_sum = wave_sum(row_sum);
    }
    const bool has = lane < d.k;
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
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
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
      row_max = wave_max(row_max);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = exp_below(p[i], row_max);
        row_sum += p[i];
      }
      row_sum = wave_sum(row_sum);
      const float inv = row_sum > 0.0f ? 1.0f / row_sum : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    const float ps = selected_score(c, xs, has, row_max, row_sum);
    float gj = 0.0f, dot = 0.0f;  // this lane's entry of the gradient
    if (c.renormalise || whole) dot = wave_sum(has ? ps * g : 0.0f);
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
      const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gj), j));
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
