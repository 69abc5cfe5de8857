// The router on gfx950: the k experts of each token and their combine
// weights from the gate logits, and the gradient of the logits.
//
// A token has a wave, or, in large batches, 16 lanes of one; lane l of L
// holds the logits of experts i * L + l, so the row is read once, coalesced,
// and stays in registers.  Choice: every key (the logit or the score, plus the
// bias) becomes an unsigned number of the
// same order; a lane sorts its keys into short lists, and k rounds find the
// largest head with a maximum over the lanes by data-parallel moves.
//
// Weights: with p the softmax or the sigmoid, a renormalised weight is
// p_j / sum_i p_i over the selected = exp(l_j - m) / sum_i exp(l_i - m) with
// l the logit (softmax) or log sigmoid(logit) = min(x, 0) - log1p(exp(-|x|))
// and m their maximum, so no logit, however far from 0, under- or overflows it.
//
// What bounds it: the instructions of the rounds, not the 16.8 MB of logits that
// 16384 tokens of 256 experts read (3.5 us at the rate of a copy): 604 vector
// instructions a token with a wave each and 8 nodes, 386 without nodes (vector
// units issuing in 90% of the time).  16384 tokens, 8 of 256 experts from 4 of 8
// nodes: 54 us with a search of all keys each round through LDS, 20.6 with
// data-parallel moves, 18.8 with sorted lists, 17.4 with the nodes' experts
// cleared through LDS instead of compared each round, 14.1 with 16 lanes a token,
// whose rounds serve four tokens.  Few tokens wait for the chain of a token's
// rounds: 5.1 us for 16, of which 4 are any launch's (the gradient's, which has no
// rounds, take 4.0).  A choice by scores has their exponentials and quotients before
// the rounds: 17.2 us there for the sigmoid and 17.6 for the softmax.
// The gradient of renormalised weights reads the k selected logits of a token, one
// by one, and writes its row, 16.8 MB there: 9.1 us, where the stores alone would
// take 3.5.  It waits for the chain of a token's ids, logits and two folds, a token
// a wave, and stores 4 bytes a lane.  That of a softmax over all experts reads the
// rows too: 12.5 us, 2.7 TB/s.
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

// The value of a key; that of a NaN, and of no expert, is -infinity.
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k <= 1u) return -INFINITY;
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// v in another lane, `other` where there is none: data-parallel moves, no LDS.
constexpr int kRowShr = 0x110, kRowRor = 0x120, kBcast15 = 0x142, kBcast31 = 0x143;
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

// Folds f over every row of 16 lanes, by rotations, or over the wave (L: 16 or
// kWave); every lane gets its result.  The order is fixed, and the same bits
// come out in every lane (the two operands of a rotation's step only swap).
template <int L, typename T, typename F>
__device__ __forceinline__ T fold(T v, T none, F f) {
  static_assert(L == 16 || L == kWave);
  if constexpr (L == 16) {
    v = f(v, moved<kRowRor + 8>(none, v));
    v = f(v, moved<kRowRor + 4>(none, v));
    v = f(v, moved<kRowRor + 2>(none, v));
    return f(v, moved<kRowRor + 1>(none, v));
  } else {
    v = f(v, moved<kRowShr + 1>(none, v));
    v = f(v, moved<kRowShr + 2>(none, v));
    v = f(v, moved<kRowShr + 4>(none, v));
    v = f(v, moved<kRowShr + 8>(none, v));
    v = f(v, moved<kBcast15, 0xa>(none, v));
    v = f(v, moved<kBcast31, 0xc>(none, v));
    if constexpr (std::is_same_v<T, float>)
      return lane_value(v, kWave - 1);
    else
      return (T)__builtin_amdgcn_readlane((int)v, kWave - 1);
  }
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return a < b ? a : b; }

template <int L>
__device__ __forceinline__ float fold_max(float v) {
  return fold<L>(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

template <int L>
__device__ __forceinline__ float fold_sum(float v) {
  return fold<L>(v, 0.0f, [](float a, float b) { return a + b; });
}

// The keys that one of a token's L lanes holds, in descending order, as lists
// of up to four with equal keys in the order of their experts; at: the
// experts, entry i starts as i * L + lane.  The token's largest key is then at
// the head of a list, and taking it moves up one list instead of searching
// all keys.
template <int V, int L>
struct Lists {
  static constexpr int kLen = V < 4 ? V : 4, kLists = V / kLen;
  uint32_t key[V], at[V];

  // Neighbours are exchanged where the second key is larger, so equal ones
  // keep their order.
  __device__ __forceinline__ void sort(int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i) at[i] = i * L + lane;
#pragma unroll
    for (int n = 0; n < V; n += kLen)
#pragma unroll
      for (int end = kLen - 1; end > 0; --end)
#pragma unroll
        for (int i = n; i < n + end; ++i) {
          const bool swap = key[i + 1] > key[i];
          const uint32_t k = key[i], a = at[i];
          key[i] = swap ? key[i + 1] : k;
          key[i + 1] = swap ? k : key[i + 1];
          at[i] = swap ? at[i + 1] : a;
          at[i + 1] = swap ? a : at[i + 1];
        }
  }

  // Takes the largest key out, of equal ones the lowest expert's, and returns
  // that expert; best becomes its key.
  __device__ __forceinline__ uint32_t take(uint32_t& best) {
    best = key[0];
#pragma unroll
    for (int n = 1; n < kLists; ++n) best = larger(best, key[n * kLen]);
    best = fold<L>(best, 0u, larger);
    // this lane's lowest expert with that key; those of a lower list are lower
    constexpr uint32_t kNone = ~0u;
    uint32_t e = kNone;
#pragma unroll
    for (int n = kLists - 1; n >= 0; --n) e = key[n * kLen] == best ? at[n * kLen] : e;
    if constexpr (L == 16) {
      e = fold<L>(e, kNone, smaller);
    } else {
      const uint64_t heads = __ballot(e != kNone);
      if ((heads & (heads - 1)) == 0)
        e = (uint32_t)__builtin_amdgcn_readlane((int)e, __builtin_ctzll(heads));
      else
        e = fold<L>(e, kNone, smaller);
    }
#pragma unroll
    for (int n = 0; n < kLists; ++n) {
      const int head = n * kLen, last = head + kLen - 1;
      const bool here = at[head] == e;
#pragma unroll
      for (int j = head; j < last; ++j) {
        key[j] = here ? key[j + 1] : key[j];
        at[j] = here ? at[j + 1] : at[j];
      }
      key[last] = here ? 0u : key[last];
    }
    return e;
  }
};

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

// Earlier accesses to LDS of this wave come before its later ones.
__device__ __forceinline__ void wave_writes_visible() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Score of the selected logit x that lane j (< k) holds, before the scale;
// lanes without a selected logit pass has = false and get 0.  row_max and
// row_sum: softmax statistics of the whole row (used without renormalising).
__device__ __forceinline__ float selected_score(const moe_router_config& c, float x, bool has,
                                                float row_max, float row_sum) {
  if (c.renormalise) {
    const float l = !has ? -INFINITY : c.score == MOE_SCORE_SIGMOID ? log_sigmoid(x) : x;
    const float m = fold_max<16>(l);
    const float e = exp_below(l, m);
    const float sum = fold_sum<16>(e);
    return sum > 0.0f ? e / sum : 0.0f;
  }
  if (!has) return 0.0f;
  if (c.score == MOE_SCORE_SIGMOID) return sigmoid(x);
  return row_sum > 0.0f ? exp_below(x, row_max) / row_sum : 0.0f;
}

// Softmax statistics of a row of which this lane holds V logits in v, which
// become exp(logit - row_max); experts past E and NaN have -infinity.
template <int V, int L>
__device__ __forceinline__ void row_statistics(float (&v)[V], float& row_max, float& row_sum) {
  row_max = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, v[i]);
  row_max = fold_max<L>(row_max);
  row_sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = exp_below(v[i], row_max);
    row_sum += v[i];
  }
  row_sum = fold_sum<L>(row_sum);
}

// A token has L lanes (16 or 64), a lane V logits (a power of two >= E / L).
// BY_SCORE: c.key is MOE_KEY_SCORE.
template <int V, int L, bool F32, bool BY_SCORE>
__global__ __launch_bounds__(kRouterWaves * kWave) void router_kernel(
    Dims d, moe_router_config c, const void* __restrict__ logits, const float* __restrict__ bias,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr int kTokens = kWave / L;      // tokens a wave
  constexpr int kRow = V * L + (V * L / 32) * 2 + 16;  // skewed, so that nodes lie in different banks
  __shared__ uint32_t s_keys[kRouterWaves][kTokens][kRow];
  const int lane = threadIdx.x % L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  uint32_t* const s_key = s_keys[wave][threadIdx.x % kWave / L];
  auto skewed = [](int e) { return e + (e >> 5) * 2; };
  int shift = L == 16 ? 4 : 6;  // log2 of the lanes a node
  while (c.nodes_per_token > 0 && d.N << shift > L) --shift;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * kTokens; t0 < d.T;
       t0 += (int64_t)gridDim.x * kRouterWaves * kTokens) {
    const int64_t at = t0 + threadIdx.x % kWave / L;
    const int64_t t = L == kWave ? t0 : std::min<int64_t>(at, d.T - 1);  // all lanes take part
    // All loads first, with no branch between them: lanes without an expert
    // load the last one's.
    float v[V];
    Lists<V, L> lists;
    uint32_t(&key)[V] = lists.key;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = load_logit<F32>(logits, t * d.E + min(i * L + lane, d.E - 1));
    float row_max = 0.0f, row_sum = 0.0f;
    if constexpr (BY_SCORE) {
      float p[V];
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = i * L + lane < d.E ? no_nan(v[i]) : -INFINITY;
      if (c.score == MOE_SCORE_SOFTMAX) {
        row_statistics<V, L>(p, row_max, row_sum);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] /= row_sum;  // > 0 where a logit is above -infinity
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = sigmoid(p[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = v[i] > -INFINITY ? p[i] : v[i];  // NaN stays NaN
    }
    if (bias != nullptr) {
      float x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = bias[min(i * L + lane, d.E - 1)];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += x[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = i * L + lane < d.E ? key_bits(v[i]) : 0;
    }
    if (c.nodes_per_token > 0) {
      // The largest two keys of each node: 1 << shift lanes scan a node's
      // consecutive experts and join what they found.  The waves of a block
      // use their own part of s_keys and do not wait for each other, only for
      // their own writes.
#pragma unroll
      for (int i = 0; i < V; ++i) s_key[skewed(i * L + lane)] = key[i];
      wave_writes_visible();
      const int share = 1 << shift, n = lane >> shift;
      const int r0 = min(n, d.N) * d.G, r1 = min(n + 1, d.N) * d.G;
      const int e0 = r0 * d.ebase + min(r0, d.erem), e1 = r1 * d.ebase + min(r1, d.erem);
      uint32_t a = 0, b = 0;
      for (int e = e0 + (lane & (share - 1)); e < e1; e += 4 * share) {
        uint32_t q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = s_key[skewed(min(e + u * share, e1 - 1))];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          q[u] = e + u * share < e1 ? q[u] : 0;
          b = larger(b, smaller(a, q[u]));
          a = larger(a, q[u]);
        }
      }
      for (int m = share >> 1; m > 0; m >>= 1) {
        const uint32_t a2 = __shfl_xor(a, m), b2 = __shfl_xor(b, m);
        b = larger(larger(b, b2), smaller(a, a2));
        a = larger(a, a2);
      }
      // two opposite infinities: the larger one decides
      const float va = key_value(a);
      const float worth = e1 - e0 < 2 || va == INFINITY ? va : va + key_value(b);
      Lists<1, L> nodes;  // entry: the node, as its first lane
      nodes.key[0] = n < d.N && (lane & (share - 1)) == 0 ? key_bits(worth) : 0;
      nodes.at[0] = lane;
      bool kept = false;
      for (int m = 0; m < c.nodes_per_token; ++m) {
        uint32_t best;
        const int taken = (int)(nodes.take(best) >> shift);  // by all lanes
        kept = kept || taken == n;
      }
      // The experts of the other nodes may not be chosen.
      if (!kept)
        for (int e = e0 + (lane & (share - 1)); e < e1; e += share) s_key[skewed(e)] = 0;
      wave_writes_visible();
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = s_key[skewed(i * L + lane)];
      wave_writes_visible();  // the next token's keys overwrite these
    }
    lists.sort(lane);
    uint32_t id = 0, taken = 0;  // lane j (< k): the j-th expert and its key
    for (int j = 0; j < d.k; ++j) {
      uint32_t best;
      const uint32_t e = lists.take(best);
      id = lane == j ? e : id;
      taken = lane == j ? best : taken;
    }
    const bool has = lane < d.k;
    float xs = key_value(taken);  // without a bias the key is the logit
    if (BY_SCORE || bias != nullptr) xs = no_nan(load_logit<F32>(logits, t * d.E + id));
    if (!BY_SCORE && c.score == MOE_SCORE_SOFTMAX && !c.renormalise) {
      // loaded again, so that the rounds above need not hold them
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * L + lane;
        v[i] = no_nan(load_logit<F32>(logits, t * d.E + min(e, d.E - 1)));
        v[i] = e < d.E ? v[i] : -INFINITY;
      }
      row_statistics<V, L>(v, row_max, row_sum);
    }
    const float p = selected_score(c, xs, has, row_max, row_sum);
    if (has && (L == kWave || at < d.T)) {
      topk_idx[t * d.k + lane] = (int32_t)id;
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
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        p[i] = e < d.E ? no_nan(load_logit<F32>(logits, t * d.E + e)) : -INFINITY;
      }
      row_statistics<V, kWave>(p, row_max, row_sum);
      const float inv = row_sum > 0.0f ? 1.0f / row_sum : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    const float ps = selected_score(c, xs, has, row_max, row_sum);
    float gj = 0.0f, dot = 0.0f;  // this lane's entry of the gradient
    if (c.renormalise || whole) dot = lane_value(fold_sum<16>(has ? ps * g : 0.0f), 0);
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

dim3 router_grid(const Dims& d, int tokens) {
  return dim3((uint32_t)std::min<int64_t>(
      ((int64_t)d.T + kRouterWaves * tokens - 1) / (kRouterWaves * tokens), kRouterMaxBlocks));
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

// Tokens up to which each gets a whole wave instead of 16 of its lanes.  Top-8,
// whole waves and 16 lanes, in us: 4096 tokens of 64 experts 4.1 and 4.1, of
// 256 in 8 nodes 6.8 and 7.6; 8192 tokens of 64 experts 5.6 and 4.1, of 128 6.0
// and 4.2, of 256 in 8 nodes 10.7 and 8.7; 16384 tokens of 64 experts 7.6 and 4.5,
// of 128 9.6 and 5.9, of 256 11.8 and 10.0, in 8 nodes 17.4 and 14.1.  More than 256
// experts would hold more than 16 keys a lane, more than 16 nodes have no lane.
constexpr int kWholeWave = 4096;

hipError_t launch_router(const Dims& d, const moe_router_config& c, const void* logits, bool f32,
                         const float* bias, int32_t* topk_idx, float* topk_w, hipStream_t s) {
  auto go = [&](auto kernel, int lanes) {
    return launch(MOE_KERNEL_ROUTER, kernel, router_grid(d, kWave / lanes),
                  dim3(kRouterWaves * kWave), 0, s, d, c, logits, bias, topk_idx, topk_w);
  };
  auto by_type = [&](auto v, auto lanes) {
    constexpr int V = decltype(v)::value, L = decltype(lanes)::value;
    if (c.key == MOE_KEY_SCORE)
      return go(f32 ? router_kernel<V, L, true, true> : router_kernel<V, L, false, true>, L);
    return go(f32 ? router_kernel<V, L, true, false> : router_kernel<V, L, false, false>, L);
  };
  if (d.T > kWholeWave && d.E <= 256 && (c.nodes_per_token == 0 || d.N <= 16)) {
    constexpr std::integral_constant<int, 16> lanes;
    if (d.E <= 64) return by_type(std::integral_constant<int, 4>(), lanes);
    if (d.E <= 128) return by_type(std::integral_constant<int, 8>(), lanes);
    return by_type(std::integral_constant<int, 16>(), lanes);
  }
  return by_experts(d.E, [&](auto v) { return by_type(v, std::integral_constant<int, kWave>()); });
}

hipError_t launch_router_grad(const Dims& d, const moe_router_config& c, const void* logits,
                              bool f32, const int32_t* topk_idx, const float* grad_w,
                              void* grad_logits, hipStream_t s) {
  return by_experts(d.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    return launch(MOE_KERNEL_ROUTER_GRAD,
                  f32 ? router_grad_kernel<V, true> : router_grad_kernel<V, false>, router_grid(d, 1),
                  dim3(kRouterWaves * kWave), 0, s, d, c, logits, topk_idx, grad_w, grad_logits);
  });
}

}  // namespace moe
