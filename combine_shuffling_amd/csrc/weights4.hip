// Packing, quantizing and unpacking of 4-bit expert weights on gfx950 (the
// layout is described in block_internal.h).  Weights are laid out once, before
// serving starts; these kernels are bound by HBM.  16 lanes take a block of 128
// weights of a row, eight consecutive ones each, and write or read its words.
#include <algorithm>

#include "block_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kUnit = 16;                             // lanes a block of 128 weights
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;      // blocks a launch

__device__ __forceinline__ uint32_t bf16_of(float f) {
  const uint32_t pair = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{f, f}, bf16x2));
  return pair & 0xffffu;
}

__device__ __forceinline__ float float_of(uint32_t bf16) { return __uint_as_float(bf16 << 16); }

// Place of a thread: eight weights k.. of row `row` (of all experts' rows).
struct At {
  int64_t row;
  int block, lane, k;
  bool live;
  __device__ __forceinline__ At(const Weights4& w, int64_t first) {
    const int64_t unit = (first * kThreads + (int64_t)blockIdx.x * kThreads + threadIdx.x) / kUnit;
    lane = threadIdx.x % kUnit;
    row = unit / w.blocks;
    block = (int)(unit - row * w.blocks);
    k = block * 128 + lane * 8;
    live = row < (int64_t)w.E * w.Z;
  }
  // The thread's word: weights 32 s + 8 g of its block, s = lane / 4 and g = lane % 4.
  __device__ __forceinline__ int64_t word(const Weights4& w) const {
    return (row * w.blocks + block) * 16 + (lane % 4) * 4 + lane / 4;
  }
  __device__ __forceinline__ int group(const Weights4& w) const { return k / w.group; }
  __device__ __forceinline__ bool first_of_group(const Weights4& w) const { return k % w.group == 0; }
  // Index of the group's scale.
  __device__ __forceinline__ int64_t scale(const Weights4& w) const {
    if (w.e2m1) return row * w.groups() + group(w);
    const int64_t e = row / w.Z;
    return (e * w.groups() + group(w)) * w.Z + (row - e * w.Z);
  }
};

// Weights in the order of a checkpoint's nibbles <-> in the order of a packed INT4 word.
__device__ __forceinline__ uint32_t int4_word(uint32_t v) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) r |= ((v >> (4 * i)) & 15u) << (4 * (i / 2) + 16 * (i % 2));
  return r;
}
__device__ __forceinline__ uint32_t int4_nibbles(uint32_t v) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) r |= ((v >> (4 * (i / 2) + 16 * (i % 2))) & 15u) << (4 * i);
  return r;
}

// A thread's eight codes (in the order of the weights) and its group's scale.
__device__ __forceinline__ void put(const Weights4& w, const At& at, uint32_t codes, uint32_t scale,
                                    uint32_t* words, void* scales) {
  words[at.word(w)] = w.e2m1 ? codes : int4_word(codes);
  if (!at.first_of_group(w)) return;
  if (w.e2m1)
    static_cast<uint8_t*>(scales)[at.scale(w)] = (uint8_t)scale;
  else
    static_cast<uint16_t*>(scales)[at.scale(w)] = (uint16_t)scale;
}

// What pads a row: weights of 0 under a finite scale.
__device__ __forceinline__ uint32_t pad_codes(const Weights4& w) { return w.e2m1 ? 0u : 0x88888888u; }
__device__ __forceinline__ uint32_t pad_scale(const Weights4& w) { return w.e2m1 ? 127u : 0u; }

__global__ __launch_bounds__(kThreads) void pack4_kernel(Weights4 w, const uint32_t* __restrict__ codes,
                                                         const void* __restrict__ given,
                                                         uint32_t* __restrict__ words,
                                                         void* __restrict__ scales, int64_t first) {
  const At at(w, first);
  if (!at.live) return;
  const uint32_t c = at.k < w.K ? codes[(at.row * w.K + at.k) / 8] : pad_codes(w);
  uint32_t s = pad_scale(w);
  if (at.first_of_group(w) && at.group(w) < w.given_groups()) {
    const int64_t from = at.row * w.given_groups() + at.group(w);
    s = w.e2m1 ? (uint32_t)static_cast<const uint8_t*>(given)[from]
               : (uint32_t)static_cast<const uint16_t*>(given)[from];
  }
  put(w, at, c, s, words, scales);
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = float_of(v[q] & 0xffffu);
    f[2 * q + 1] = __uint_as_float(v[q] & 0xffff0000u);
  }
}

__global__ __launch_bounds__(kThreads) void quantize4_kernel(Weights4 w,
                                                             const uint16_t* __restrict__ from,
                                                             uint32_t* __restrict__ words,
                                                             void* __restrict__ scales,
                                                             int64_t first) {
  const At at(w, first);
  float f[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = 0.0f;
  const bool in = at.live && at.k < w.K;
  if (in) load8(from + at.row * w.K + at.k, f);
  // The largest magnitude of the group, as the bits of |w|: they order as the values do, and
  // those of infinities and NaNs are above all others.
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) most = max(most, __float_as_uint(f[q]) & 0x7fffffffu);
  for (int d = 1; d < w.group / 8; d <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, d));
  if (!at.live) return;
  const bool finite = most < 0x7f800000u;
  const float amax = __uint_as_float(most);
  uint32_t codes = 0, scale;
  if (w.e2m1) {
    int e = 0;
    if (finite && most != 0u) {
      int p;
      const float m = frexpf(amax, &p);              // amax = m 2^p, m in [0.5, 1)
      e = min(max(p - 3 + (m > 0.75f ? 1 : 0), -127), 127);  // the smallest with amax <= 6 2^e
    }
    scale = finite ? (uint32_t)(e + 127) : 255u;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float v = finite ? ldexpf(fabsf(f[q]), -e) : 0.0f;
      uint32_t c = (uint32_t)(v > 0.25f) + (v >= 0.75f) + (v > 1.25f) + (v >= 1.75f) + (v > 2.5f) +
                   (v >= 3.5f) + (v > 5.0f);
      if (finite) c |= __float_as_uint(f[q]) >> 31 << 3;
      codes |= c << (4 * q);
    }
  } else {
    scale = finite ? bf16_of(amax / 7.0f) : 0x7fc0u;
    const float s = float_of(scale);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float v = finite && s > 0.0f ? fminf(fmaxf(rintf(f[q] / s), -8.0f), 7.0f) : 0.0f;
      codes |= (uint32_t)((int)v + 8) << (4 * q);
    }
  }
  put(w, at, in ? codes : pad_codes(w), at.k < w.K || !at.first_of_group(w) ? scale : pad_scale(w), words,
      scales);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void unpack4_kernel(Weights4 w,
                                                           const uint32_t* __restrict__ words,
                                                           const void* __restrict__ scales,
                                                           void* __restrict__ to, int64_t first) {
  const At at(w, first);
  if (!at.live || at.k >= w.K) return;
  const uint32_t word = words[at.word(w)];
  float f[8];
  if (w.e2m1) {
    const uint32_t s = static_cast<const uint8_t*>(scales)[at.scale(w)];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t c = (word >> (4 * q)) & 15u, e = (c >> 1) & 3u;
      // two bits of exponent (bias 1), one of mantissa
      const float m = e == 0 ? 0.5f * (float)(c & 1u) : ldexpf(1.0f + 0.5f * (float)(c & 1u), (int)e - 1);
      const float v = c & 8u ? -m : m;
      f[q] = s == 255u ? __uint_as_float(0x7fc00000u) : ldexpf(v, (int)s - 127);
    }
  } else {
    const float s = float_of(static_cast<const uint16_t*>(scales)[at.scale(w)]);
    const uint32_t n = int4_nibbles(word);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = s * (float)((int)((n >> (4 * q)) & 15u) - 8);
  }
  const int64_t chunk = (at.row * w.K + at.k) / 8;
  if constexpr (F32) {
    f32x4* o = static_cast<f32x4*>(to) + chunk * 2;
    o[0] = f32x4{f[0], f[1], f[2], f[3]};
    o[1] = f32x4{f[4], f[5], f[6], f[7]};
  } else {
    u32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = bf16_of(f[2 * q]) | bf16_of(f[2 * q + 1]) << 16;
    static_cast<u32x4*>(to)[chunk] = r;
  }
}

template <typename F>
hipError_t in_ranges(const Weights4& w, F f) {
  const int64_t total = ((int64_t)w.E * w.Z * w.blocks * kUnit + kThreads - 1) / kThreads;
  for (int64_t b = 0; b < total; b += kMaxBlocks) {
    f(dim3((uint32_t)std::min(total - b, kMaxBlocks)), b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_pack4(const Weights4& w, const uint8_t* codes, const void* scales, void* packed,
                        hipStream_t s) {
  return in_ranges(w, [&](dim3 blocks, int64_t first) {
    pack4_kernel<<<blocks, kThreads, 0, s>>>(w, reinterpret_cast<const uint32_t*>(codes), scales,
                                             static_cast<uint32_t*>(packed),
                                             static_cast<char*>(packed) + w.codes_bytes(), first);
  });
}

hipError_t launch_quantize4(const Weights4& w, const uint16_t* from, void* packed, hipStream_t s) {
  return in_ranges(w, [&](dim3 blocks, int64_t first) {
    quantize4_kernel<<<blocks, kThreads, 0, s>>>(w, from, static_cast<uint32_t*>(packed),
                                                 static_cast<char*>(packed) + w.codes_bytes(), first);
  });
}

hipError_t launch_unpack4(const Weights4& w, const void* packed, void* to, bool f32, hipStream_t s) {
  return in_ranges(w, [&](dim3 blocks, int64_t first) {
    auto go = [&](auto kernel) {
      kernel<<<blocks, kThreads, 0, s>>>(w, static_cast<const uint32_t*>(packed),
                                         static_cast<const char*>(packed) + w.codes_bytes(), to, first);
    };
    f32 ? go(unpack4_kernel<true>) : go(unpack4_kernel<false>);
  });
}

}  // namespace moe
