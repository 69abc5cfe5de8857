// Packing, quantizing and unpacking of 4-bit expert weights on gfx950 (the
// layout is described in block_internal.h).  Weights are laid out once, before
// serving starts.  A wave takes a tile of 16 rows by 128 along K, a lane the 16 bytes
// that it has in the layout: whole lines on the packed side, 64 bytes (of codes, 16) of
// each of 16 rows at a time on the other.  64 x 2048 x 2048 weights, by format, of a
// copy's 4.7 TB/s: packing 92 to 128 us (2.4 to 3.0 TB/s), quantizing 192 to 224 (3.1 to 3.5),
// unpacking to bf16 148 to 176 (3.9 to 4.6); groups of 32 take the longest.
#include <algorithm>

#include "block_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;  // blocks a launch

__device__ __forceinline__ uint32_t bf16_of(float f) {
  const uint32_t pair = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{f, f}, bf16x2));
  return pair & 0xffffu;
}

__device__ __forceinline__ float float_of(uint32_t bf16) { return __uint_as_float(bf16 << 16); }

// A lane's place: its piece of 16 bytes, row i of a tile, weights 32 s + 8 g + 0..7 of the tile's
// block of 128.
struct At {
  int64_t piece, tile, row;  // the row of all experts' rows, unpadded
  int i, g, k0;              // k0: the block's first weight
  bool live, in_rows;
  __device__ __forceinline__ At(const Weights4& w, int64_t first) {
    piece = (first + blockIdx.x) * kThreads + threadIdx.x;
    tile = piece / kWave;
    const int lane = threadIdx.x % kWave;
    i = lane % 16;
    g = lane / 16;
    const int64_t rows16 = tile / w.blocks;
    k0 = (int)(tile - rows16 * w.blocks) * 128;
    const int64_t e = rows16 / w.tiles;
    const int r = (int)(rows16 - e * w.tiles) * 16 + i;
    live = e < w.E;
    in_rows = live && r < w.Z;
    row = e * w.Z + r;
  }
  __device__ __forceinline__ int k(int s) const { return k0 + 32 * s + 8 * g; }
  // Index of the scale of weights k(s).
  __device__ __forceinline__ int64_t scale(const Weights4& w, int s) const {
    const int groups = 128 / w.group, q = s * 32 / w.group, beside = w.beside();
    return tile * 16 * groups + q / beside * 16 * beside + i * beside + q % beside;
  }
  // Whether this lane writes that scale, for its group.
  __device__ __forceinline__ bool writes(const Weights4& w, int s) const {
    return g == 0 && s * 32 % w.group == 0;
  }
};

// Weights in the order of a checkpoint's nibbles <-> in the order of a packed INT4 word.
__device__ __forceinline__ uint32_t int4_word(uint32_t v) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) r |= ((v >> (4 * i)) & 15u) << (4 * (i / 2) + 16 * (i % 2));
  return __builtin_rotateleft32(r, 3);
}
__device__ __forceinline__ uint32_t int4_nibbles(uint32_t v) {
  uint32_t r = 0;
  v = __builtin_rotateright32(v, 3);
#pragma unroll
  for (int i = 0; i < 8; ++i) r |= ((v >> (4 * (i / 2) + 16 * (i % 2))) & 15u) << (4 * i);
  return r;
}

__device__ __forceinline__ void put_scale(const Weights4& w, const At& at, int s, uint32_t scale,
                                          void* scales) {
  if (!at.writes(w, s)) return;
  if (w.e2m1)
    static_cast<uint8_t*>(scales)[at.scale(w, s)] = (uint8_t)scale;
  else
    static_cast<uint16_t*>(scales)[at.scale(w, s)] = (uint16_t)scale;
}

// What pads rows and K: weights of 0 under a finite scale (codes in a checkpoint's order).
__device__ __forceinline__ uint32_t pad_codes(const Weights4& w) { return w.e2m1 ? 0u : 0x88888888u; }
__device__ __forceinline__ uint32_t pad_scale(const Weights4& w) { return w.e2m1 ? 127u : 0u; }

__global__ __launch_bounds__(kThreads) void pack4_kernel(Weights4 w, const uint32_t* __restrict__ codes,
                                                         const void* __restrict__ given,
                                                         u32x4* __restrict__ pieces,
                                                         void* __restrict__ scales, int64_t first) {
  const At at(w, first);
  if (!at.live) return;
  u32x4 piece;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const bool in = at.in_rows && at.k(s) < w.K;
    const uint32_t c = in ? codes[(at.row * w.K + at.k(s)) / 8] : pad_codes(w);
    piece[s] = w.e2m1 ? c : int4_word(c);
    uint32_t scale = pad_scale(w);
    const int group = (at.k0 + 32 * s) / w.group;
    if (at.writes(w, s) && at.in_rows && group < w.given_groups()) {
      const int64_t from = at.row * w.given_groups() + group;
      scale = w.e2m1 ? (uint32_t)static_cast<const uint8_t*>(given)[from]
                     : (uint32_t)static_cast<const uint16_t*>(given)[from];
    }
    put_scale(w, at, s, scale, scales);
  }
  pieces[at.piece] = piece;
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
                                                             u32x4* __restrict__ pieces,
                                                             void* __restrict__ scales,
                                                             int64_t first) {
  const At at(w, first);
  float f[4][8];
  // The largest magnitude of each group, as the bits of |w|: they order as the values do, and
  // those of infinities and NaNs are above all others.
  uint32_t most[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[s][q] = 0.0f;
    if (at.in_rows && at.k(s) < w.K) load8(from + at.row * w.K + at.k(s), f[s]);
    most[s] = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) most[s] = max(most[s], __float_as_uint(f[s][q]) & 0x7fffffffu);
    most[s] = max(most[s], (uint32_t)__shfl_xor((int)most[s], 16));
    most[s] = max(most[s], (uint32_t)__shfl_xor((int)most[s], 32));
  }
  if (!at.live) return;
  if (w.group >= 64) {
    most[0] = most[1] = max(most[0], most[1]);
    most[2] = most[3] = max(most[2], most[3]);
  }
  if (w.group == 128) most[0] = most[1] = most[2] = most[3] = max(most[0], most[2]);
  u32x4 piece;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const bool finite = most[s] < 0x7f800000u;
    const float amax = __uint_as_float(most[s]);
    uint32_t codes = 0, scale;
    if (w.e2m1) {
      int e = 0;
      if (finite && most[s] != 0u) {
        int p;
        const float m = frexpf(amax, &p);                      // amax = m 2^p, m in [0.5, 1)
        e = min(max(p - 3 + (m > 0.75f ? 1 : 0), -127), 127);  // the smallest with amax <= 6 2^e
      }
      scale = finite ? (uint32_t)(e + 127) : 255u;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float v = finite ? ldexpf(fabsf(f[s][q]), -e) : 0.0f;
        uint32_t c = (uint32_t)(v > 0.25f) + (v >= 0.75f) + (v > 1.25f) + (v >= 1.75f) + (v > 2.5f) +
                     (v >= 3.5f) + (v > 5.0f);
        if (finite) c |= __float_as_uint(f[s][q]) >> 31 << 3;
        codes |= c << (4 * q);
      }
    } else {
      scale = finite ? bf16_of(amax / 7.0f) : 0x7fc0u;
      const float unit = float_of(scale);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float v = finite && unit > 0.0f ? fminf(fmaxf(rintf(f[s][q] / unit), -8.0f), 7.0f) : 0.0f;
        codes |= (uint32_t)((int)v + 8) << (4 * q);
      }
    }
    const bool in = at.in_rows && at.k(s) < w.K;
    if (!in) codes = pad_codes(w);
    piece[s] = w.e2m1 ? codes : int4_word(codes);
    put_scale(w, at, s, at.in_rows && at.k0 + 32 * s < w.K ? scale : pad_scale(w), scales);
  }
  pieces[at.piece] = piece;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void unpack4_kernel(Weights4 w,
                                                           const u32x4* __restrict__ pieces,
                                                           const void* __restrict__ scales,
                                                           void* __restrict__ to, int64_t first) {
  const At at(w, first);
  if (!at.in_rows) return;
  const u32x4 piece = pieces[at.piece];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (at.k(s) >= w.K) break;
    float f[8];
    if (w.e2m1) {
      const uint32_t scale = static_cast<const uint8_t*>(scales)[at.scale(w, s)];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t c = (piece[s] >> (4 * q)) & 15u, e = (c >> 1) & 3u;
        // two bits of exponent (bias 1), one of mantissa
        const float m = e == 0 ? 0.5f * (float)(c & 1u) : ldexpf(1.0f + 0.5f * (float)(c & 1u), (int)e - 1);
        const float v = c & 8u ? -m : m;
        f[q] = scale == 255u ? __uint_as_float(0x7fc00000u) : ldexpf(v, (int)scale - 127);
      }
    } else {
      const float scale = float_of(static_cast<const uint16_t*>(scales)[at.scale(w, s)]);
      const uint32_t n = int4_nibbles(piece[s]);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = scale * (float)((int)((n >> (4 * q)) & 15u) - 8);
    }
    const int64_t chunk = (at.row * w.K + at.k(s)) / 8;
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
}

template <typename F>
hipError_t in_ranges(const Weights4& w, F f) {
  const int64_t total = ((int64_t)w.E * w.tiles * w.blocks * kWave + kThreads - 1) / kThreads;
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
                                             static_cast<u32x4*>(packed),
                                             static_cast<char*>(packed) + w.codes_bytes(), first);
  });
}

hipError_t launch_quantize4(const Weights4& w, const uint16_t* from, void* packed, hipStream_t s) {
  return in_ranges(w, [&](dim3 blocks, int64_t first) {
    quantize4_kernel<<<blocks, kThreads, 0, s>>>(w, from, static_cast<u32x4*>(packed),
                                                 static_cast<char*>(packed) + w.codes_bytes(), first);
  });
}

hipError_t launch_unpack4(const Weights4& w, const void* packed, void* to, bool f32, hipStream_t s) {
  return in_ranges(w, [&](dim3 blocks, int64_t first) {
    auto go = [&](auto kernel) {
      kernel<<<blocks, kThreads, 0, s>>>(w, static_cast<const u32x4*>(packed),
                                         static_cast<const char*>(packed) + w.codes_bytes(), to, first);
    };
    f32 ? go(unpack4_kernel<true>) : go(unpack4_kernel<false>);
  });
}

}  // namespace moe
