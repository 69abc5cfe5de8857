// The experts' matrix products on gfx950, forward and backward: for every
// expert e with receive rows [off[e], off[e + 1])
//   rows       z = x w[e]^T (+ bias, activation, residual)  contracts over K
//   rows grad  gx = gz w[e]                                 contracts over Z
//   wgrad      gw[e] = gz^T x                               contracts over e's rows
//
// One block computes one BM x BN tile of one expert's result with bf16 matrix
// instructions (16x16x32) and float32 accumulators that stay in registers.
// Per step of 64 along the contraction both operands' tiles are loaded
// straight into LDS (buffer loads with an LDS destination), two stages deep:
// the loads of the next step are in flight while this one is multiplied.
//
// An operand whose memory is contiguous along the contraction (x and w of
// `rows`, gz of `rows grad`) is kept as rows of 64 values (128 bytes), one
// 16-byte read per lane and fragment; an operand that is contiguous across it
// (w of `rows grad`, both of wgrad) as 64 rows along the contraction, read
// through the transposing LDS read.  Both layouts are swizzled so that the
// lanes of a read fall into different banks; since a load to LDS writes lanes
// one after another, the swizzle permutes which global chunk a lane loads.
//
// Rows of different experts never share a tile, and the counts are only
// known on the device: expert e's row tiles take the slots from
// off[e] / BM + e on, which is at least ceil(rows / BM) slots each and
// rows / BM + E in all; a block finds its expert by searching off and leaves
// if its slot is not used.
//
// Loads go through buffer descriptors that end with the operand's rows, so
// rows past the end read as zeros; columns past the width of a transposed
// operand give results that are not stored.  Chunks past the end of a
// contiguous contraction are sent past the descriptor's end, so that they
// read as zeros on both sides.
#include <algorithm>
#include <type_traits>

#include "layer_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
#define MOE_LDS __attribute__((address_space(3)))

constexpr int kBK = 32;                   // contraction step: 64 bytes of bf16
constexpr int kBufferFormat = 0x00020000; // raw buffer descriptor, word 3 (gfx9 family)
constexpr uint32_t kPast = 0x80000000u;   // an offset past every descriptor's end
constexpr int kXcds = 8;
constexpr int64_t kMaxTileBlocks = (int64_t)1 << 22;  // blocks a launch (work-items are counted in 32 bits)

// Two floats to bf16, round to nearest even, NaN stays NaN (one instruction).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(v[q] << 16);
    f[2 * q + 1] = __uint_as_float(v[q] & 0xffff0000u);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  u32x4 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r[q] = bf16_pair(f[2 * q], f[2 * q + 1]);
  return r;
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// Descriptor of the `bytes` bytes at p, both the same in every lane (said
// outright: a descriptor that the compiler takes for divergent costs a loop
// over the lanes around every load).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_buffer(const char* p, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint64_t v = (uint64_t)uniform((uint32_t)(u >> 32)) << 32 | uniform((uint32_t)u);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(v), 0, (int)uniform(bytes),
                                           kBufferFormat);
}

// ---- activations

__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }

__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// z := act(z), one choice for eight values.
__device__ __forceinline__ void act_values(int act, float (&z)[8]) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] = z[q] < 0.0f ? 0.0f : z[q];
      break;
    case MOE_ACT_SILU:
    case MOE_ACT_SWIGLU:
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] *= logistic(z[q]);
      break;
    case MOE_ACT_GELU:
    case MOE_ACT_GEGLU:
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] *= normal_cdf(z[q]);
      break;
    default: break;
  }
}

// value := act(z), slope := act'(z).
__device__ __forceinline__ void act_slopes(int act, const float (&z)[8], float (&value)[8],
                                           float (&slope)[8]) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        slope[q] = z[q] > 0.0f ? 1.0f : 0.0f;
        value[q] = z[q] < 0.0f ? 0.0f : z[q];
      }
      break;
    case MOE_ACT_SILU:
    case MOE_ACT_SWIGLU:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float p = logistic(z[q]);
        value[q] = z[q] * p;
        slope[q] = p * (1.0f + z[q] * (1.0f - p));
      }
      break;
    case MOE_ACT_GELU:
    case MOE_ACT_GEGLU:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float p = normal_cdf(z[q]);
        value[q] = z[q] * p;
        slope[q] = p + z[q] * 0.3989422804014327f * __expf(-0.5f * z[q] * z[q]);
      }
      break;
    default:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        value[q] = z[q];
        slope[q] = 1.0f;
      }
  }
}

// ---- which expert and rows a slot of BM rows stands for

struct Segment {
  int e;      // expert
  int row;    // first row
  int rows;   // rows of the tile (<= 0: the slot is not used)
  int left;   // rows of the expert from `row` on
};

// The last expert whose first slot, off[e] / BM + e, is <= slot.  Two rounds
// of one load a lane: every ceil(E / 64)-th expert, then those in between.
__device__ __forceinline__ Segment find_segment(const int32_t* off, int E, int slot, int bm) {
  const int lane = threadIdx.x & (kWave - 1);
  const int step = (E + kWave - 1) / kWave;
  const int e1 = lane * step;
  const bool in1 = e1 < E && off[min(e1, E)] / bm + e1 <= slot;
  int e = (__popcll(__ballot(in1)) - 1) * step;  // lane 0 is always in
  if (step > 1) {
    const int e2 = e + lane;
    const bool in2 = lane < step && e2 < E && off[min(e2, E)] / bm + e2 <= slot;
    e += __popcll(__ballot(in2)) - 1;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  Segment s;
  const int o0 = off[e], o1 = off[e + 1];
  s.e = e;
  s.row = o0 + (slot - (o0 / bm + e)) * bm;
  s.left = o1 - s.row;
  s.rows = min(s.left, bm);
  return s;
}

// Which tile of a [mtiles, ntiles] grid (or of a row of such grids, one an
// expert) a block computes.  The tiles are cut into groups of about kGroup x
// kGroup result elements, and the groups are dealt to the XCDs in turn (as the hardware deals
// the blocks): the blocks that run on an XCD at one time share few rows and
// columns of the operands, which they find in that XCD's L2, and neighbouring
// groups run on the other XCDs, which find them in the cache behind it.
struct Tile {
  int grid, m, n;
  bool live;
};

constexpr int kGroup = 1024;

template <int BM, int BN>
struct TileGrid {
  static constexpr int kGroupM = kGroup / BM, kGroupN = kGroup / BN, kTiles = kGroupM * kGroupN;
  int grids, mtiles, ntiles;
  int mgroups, ngroups;

  TileGrid(int grids_, int mtiles_, int ntiles_)
      : grids(grids_), mtiles(mtiles_), ntiles(ntiles_),
        mgroups((mtiles_ + kGroupM - 1) / kGroupM), ngroups((ntiles_ + kGroupN - 1) / kGroupN) {}
  // Blocks of all launches together.
  int64_t blocks() const {
    const int64_t groups = (int64_t)grids * mgroups * ngroups;
    return (groups + kXcds - 1) / kXcds * kXcds * kTiles;
  }
  __device__ __forceinline__ Tile at(int64_t block) const {
    const int64_t i = block / kXcds;
    const int64_t group = i / kTiles * kXcds + block % kXcds;
    const int in = (int)(i % kTiles);
    const int per = mgroups * ngroups;
    Tile t;
    t.grid = (int)(group / per);
    const int g = (int)(group % per);
    t.m = g / ngroups * kGroupM + in / kGroupN;
    t.n = g % ngroups * kGroupN + in % kGroupN;
    t.live = t.grid < grids && t.m < mtiles && t.n < ntiles;
    return t;
  }
};

// ---- the tile product

// One operand's tile: where its bytes are and how far they go.
struct Operand {
  const char* base;   // row 0, contraction 0
  uint32_t ld;        // bytes between rows of memory
  uint32_t bytes;     // contiguous contraction: bytes from base to the end of the tile's rows
};

template <int BM_, int BN_, int WM_, int WN_, bool AT_, bool BT_, bool GATED_>
struct TileProduct {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr bool AT = AT_, BT = BT_, GATED = GATED_;
  static constexpr int kNW = WM * WN, kThreads = kNW * kWave;
  static constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 16, NJ = TN / 16;
  static constexpr int kABytes = BM * kBK * 2, kBBytes = BN * kBK * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 3;
  static constexpr int kLds = kStages * kStage;
  static constexpr int QA = kABytes / 1024 / kNW, QB = kBBytes / 1024 / kNW;  // loads a wave and stage
  static_assert(QA * kNW * 1024 == kABytes && QB * kNW * 1024 == kBBytes);
  static_assert(BT || TN == 64, "the permuted columns of a wave are 64 wide");

  // Contiguous contraction: LDS row r (64 bytes, 4 chunks) holds chunk
  // p ^ swizzle(r) at position p.  A's rows are read in order; B's in the
  // order of the permuted columns (rows i % 4 + 16 * (i / 4) for lane i), so
  // each has the swizzle that spreads its own eight consecutive lanes over
  // all banks.
  template <bool B>
  static __device__ __forceinline__ int swizzle(int r) {
    return B ? ((r >> 1) & 1) | ((r >> 4) & 1) << 1 : (r >> 1) & 3;
  }
  // Transposed: LDS row kr (along the contraction) of W columns; the 32-byte
  // block b of a row sits at position b ^ spread(kr).
  template <int W>
  static __device__ __forceinline__ int spread(int kr) {
    return ((kr & 3) | ((kr >> 3) & 3) << 2) & (W / 16 - 1);
  }
  // Byte offset in memory of a lane's 16 bytes for the wave's q-th load.
  template <int W>
  static __device__ __forceinline__ uint32_t offset_t(uint32_t ld, int wave, int lane, int q) {
    constexpr int per = W / 8;       // 16-byte positions a row
    const int pos = (q * kNW + wave) * 64 + lane;
    const int kr = pos / per, p = pos % per;
    return kr * ld + ((((p >> 1) ^ spread<W>(kr)) << 1) | (p & 1)) * 16;
  }

  // Memory row of B's LDS row r.  Gated: a wave's 64 rows are 32 of the gate
  // and 32 of the up projection, in the order that puts 8 consecutive columns
  // of both into one lane.
  static __device__ __forceinline__ int b_row(int r, int gate_up) {
    if constexpr (!GATED) return r;
    const int slab = r / 64, q = (r >> 4) & 3, jj = (r >> 2) & 3;
    return slab * 32 + q * 8 + (jj & 1) * 4 + (r & 3) + (jj >> 1) * gate_up;
  }

  struct Fragments {
    bf16x8 a[MI], b[NJ];
  };

  f32x4 acc[MI][NJ];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // acc += A B over `len` contraction elements.  rows: result rows that are
  // wanted (the others' products are skipped, 16 rows at a time).  gate_up:
  // memory rows from the gate's to the up projection's row (gated only).
  //
  // While the fragments of step s (in registers) are multiplied, those of
  // step s + 1 are read from LDS and the loads of steps s + 2 and s + 3 are
  // under way.  One barrier a step: before it a wave waits for its own
  // fragments of step s (so stage s is free after it, for step s + 3) and for
  // its own loads of step s + 1 (so they can be read after it).  Steps past
  // the end load zeros through empty descriptors, which keeps the number of
  // loads under way the same in every step.
  __device__ __forceinline__ void run(const Operand& a, const Operand& b, int len, int rows,
                                      int gate_up, char* lds) {
    const int m0 = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) / WN * TM;
    const int used = min(max((rows - m0 + 15) / 16, 0), MI);
    if (used == MI)
      sweep<true>(a, b, len, MI, gate_up, lds);
    else
      sweep<false>(a, b, len, used, gate_up, lds);
  }

  template <bool FULL>
  __device__ __forceinline__ void sweep(const Operand& a, const Operand& b, int len, int used,
                                        int gate_up, char* lds) {
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    uint32_t va[QA], vb[QB];
    int ca[QA], cb[QB];  // chunk of the step a lane loads (contiguous contraction)
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int r = (q * kNW + wave) * 16 + lane / 4;
      ca[q] = AT ? 0 : (lane & 3) ^ swizzle<false>(r);
      va[q] = AT ? offset_t<BM>(a.ld, wave, lane, q) : (uint32_t)r * a.ld + ca[q] * 16;
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int r = (q * kNW + wave) * 16 + lane / 4;
      cb[q] = BT ? 0 : (lane & 3) ^ swizzle<true>(r);
      vb[q] = BT ? offset_t<BN>(b.ld, wave, lane, q)
                 : (uint32_t)b_row(r, gate_up) * b.ld + cb[q] * 16;
    }
    const int m0 = wave / WN * TM, n0 = wave % WN * TN;
    const int steps = (len + kBK - 1) / kBK;
    auto load = [&](int step, char* to) {
      const int done = step * kBK, left = len - done;
      issue<AT, QA>(a, va, ca, done, left, to + wave * 1024);
      issue<BT, QB>(b, vb, cb, done, left, to + kABytes + wave * 1024);
    };
    auto read = [&](Fragments& f, const char* from) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) f.b[j] = fragment<BT, true, BN>(from + kABytes, n0, j, lane);
#pragma unroll
      for (int i = 0; i < MI; ++i)
        if (FULL || i < used) f.a[i] = fragment<AT, false, BM>(from, m0, i, lane);
    };
    int put = 0, get = kStage;  // LDS offsets of the next stage to load and to read
    auto step = [&](int s, const Fragments& now, Fragments& next) {
      wait_and_meet<QA + QB>();
      refill(load, read, s + 3, next, lds + put, lds + get);
      put = put == (kStages - 1) * kStage ? 0 : put + kStage;
      get = get == (kStages - 1) * kStage ? 0 : get + kStage;
#pragma unroll
      for (int i = 0; i < MI; ++i)
        if (FULL || i < used)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.b[j], now.a[i], acc[i][j], 0, 0, 0);
      if constexpr (FULL) interleave();
      __builtin_amdgcn_sched_barrier(0);
    };
    load(0, lds);
    load(1, lds + kStage);
    load(2, lds + 2 * kStage);
    wait_and_meet<2 * (QA + QB)>();
    Fragments f0{}, f1{};
    read(f0, lds);
    for (int s = 0; s < steps; s += 2) {
      step(s, f0, f1);
      if (s + 1 < steps) step(s + 1, f1, f0);
    }
    wait_and_meet<0>();  // nothing may land in LDS after the block has ended
  }

  // The loads of a later step and the reads of the next.  The two stages are
  // different ones, and saying so (restrict) matters: where the compiler sees
  // that a read from LDS may touch what a load to LDS writes, it waits for
  // every load under way before the read.
  template <typename L, typename R>
  static __device__ __forceinline__ void refill(const L& load, const R& read, int step,
                                                Fragments& next, char* __restrict__ to,
                                                const char* __restrict__ from) {
    load(step, to);
    read(next, from);
  }

  // Waits until at most N of this wave's loads to LDS and none of its LDS
  // reads are under way, then for the block's other waves.
  template <int N>
  static __device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // Asks the scheduler to start with products (whose fragments have been
  // waited for) and to spread the loads and the reads over the rest.
  static __device__ __forceinline__ void interleave() {
    constexpr int loads = QA + QB, reads = MI * (AT ? 2 : 1) + NJ * (BT ? 2 : 1);
    constexpr int products = MI * NJ, each = (products - 2) / reads;
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);  // matrix instructions
#pragma unroll
    for (int i = 0; i < reads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      if (i < loads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // load
      __builtin_amdgcn_sched_group_barrier(0x008, each, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, products - 2 - reads * each, 0);
  }

  template <bool T, int Q>
  static __device__ __forceinline__ void issue(const Operand& o, const uint32_t (&v)[Q],
                                               const int (&c)[Q], int done, int left, char* at) {
    const char* base;
    uint32_t bytes;
    if constexpr (T) {
      base = o.base + (int64_t)done * o.ld;
      bytes = (uint32_t)max(min(left, kBK), 0) * o.ld;
      bytes = bytes > o.bytes ? bytes - o.bytes : 0;  // o.bytes: the tile's first column
    } else {
      base = o.base + (int64_t)done * 2;
      bytes = left > 0 && o.bytes > (uint32_t)done * 2 ? o.bytes - done * 2 : 0;
    }
    const __amdgpu_buffer_rsrc_t r = uniform_buffer(base, bytes);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      uint32_t off = v[q];
      if constexpr (!T)
        if (left < kBK) off = c[q] * 8 < left ? off : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void*)(at + q * kNW * 1024), 16, off, 0, 0,
                                               0);
    }
  }

  template <bool T, bool B, int W>
  static __device__ __forceinline__ bf16x8 fragment(const char* tile, int first, int f, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (T) {
      const int kr = g * 8 + (i >> 2);
      const char* p = tile + kr * (W * 2) + (((first / 16 + f) ^ spread<W>(kr)) << 5) + (i & 3) * 8;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(p + 4 * W * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = B ? first + (i >> 2) * 16 + f * 4 + (i & 3) : first + f * 16 + i;
      const char* p = tile + r * 64 + ((g ^ swizzle<B>(r)) << 4);
      return *reinterpret_cast<const bf16x8*>(p);
    }
  }
};

// A lane of acc[i][j] holds result row (first row of the wave) + i * 16 + lane % 16
// and four consecutive columns, lane / 16 * 4 + 0..3 of the fragment.  In the
// row product the fragment's columns are spread so that a lane's NJ * 4
// columns are consecutive: lane / 16 * 16 + j * 4 + 0..3 of the wave's 64
// (gated: lane / 16 * 8 + (j & 1) * 4 of its 32, j >> 1 the gate or up).

// ---- rows: y = act(x w^T + bias) + residual

template <typename P>
__global__ __launch_bounds__(P::kThreads, 2) void expert_rows_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ a,
    const char* __restrict__ w, const float* __restrict__ bias,
    const uint16_t* __restrict__ residual, uint16_t* __restrict__ y, uint16_t* __restrict__ pre,
    TileGrid<P::BM, P::BN> grid, int64_t base) {
  __shared__ __align__(1024) char lds[P::kLds];
  constexpr int kCols = P::GATED ? P::BN / 2 : P::BN;  // columns of y a tile
  const Tile tile = grid.at(base + blockIdx.x);
  if (!tile.live) return;
  const Segment s = find_segment(off, x.E, tile.m, P::BM);
  if (s.rows <= 0) return;
  const int n0 = tile.n * kCols;
  const uint32_t ld = (uint32_t)x.K * 2;
  Operand oa{a + (int64_t)s.row * ld, ld, (uint32_t)s.rows * ld};
  Operand ob{w + ((int64_t)s.e * x.Z + n0) * ld, ld, (uint32_t)(x.Z - n0) * ld};
  P p;
  p.clear();
  p.run(oa, ob, x.K, s.rows, x.N, lds);

  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int g = lane >> 4;
  const int m0 = wave / P::WN * P::TM + (lane & 15);
  const int c0 = n0 + wave % P::WN * (P::GATED ? 32 : 64) + g * (P::GATED ? 8 : 16);
  float bz[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) bz[q] = 0.0f;
  if (bias != nullptr) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = P::GATED ? c0 : c0 + h * 8;
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
#pragma unroll
  for (int i = 0; i < P::MI; ++i) {
    const int m = m0 + i * 16;
    if (m >= s.rows) continue;
    const int64_t row = s.row + m;
    float z[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) z[j * 4 + q] = p.acc[i][j][q] + bz[j * 4 + q];
    if constexpr (P::GATED) {
      if (c0 >= x.N) continue;
      float gate[8], up[8], out[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        out[q] = gate[q] = z[q];
        up[q] = z[8 + q];
      }
      act_values(x.act, out);
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] *= up[q];
      if (pre != nullptr) {
        *reinterpret_cast<u32x4*>(pre + row * x.Z + c0) = pack8(gate);
        *reinterpret_cast<u32x4*>(pre + row * x.Z + x.N + c0) = pack8(up);
      }
      if (residual != nullptr) {
        float r[8];
        unpack8(*reinterpret_cast<const u32x4*>(residual + row * x.N + c0), r);
#pragma unroll
        for (int q = 0; q < 8; ++q) out[q] += r[q];
      }
      *reinterpret_cast<u32x4*>(y + row * x.N + c0) = pack8(out);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = c0 + h * 8;
        if (col >= x.N) continue;
        float out[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) out[q] = z[h * 8 + q];
        if (pre != nullptr) *reinterpret_cast<u32x4*>(pre + row * x.Z + col) = pack8(out);
        act_values(x.act, out);
        if (residual != nullptr) {
          float r[8];
          unpack8(*reinterpret_cast<const u32x4*>(residual + row * x.N + col), r);
#pragma unroll
          for (int q = 0; q < 8; ++q) out[q] += r[q];
        }
        *reinterpret_cast<u32x4*>(y + row * x.N + col) = pack8(out);
      }
    }
  }
}

// ---- rows grad: gx = gz w

template <typename P>
__global__ __launch_bounds__(P::kThreads, 2) void expert_rows_grad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ gz,
    const char* __restrict__ w, uint16_t* __restrict__ gx, TileGrid<P::BM, P::BN> grid, int64_t base) {
  __shared__ __align__(1024) char lds[P::kLds];
  const Tile tile = grid.at(base + blockIdx.x);
  if (!tile.live) return;
  const Segment s = find_segment(off, x.E, tile.m, P::BM);
  if (s.rows <= 0) return;
  const int n0 = tile.n * P::BN;
  const uint32_t lda = (uint32_t)x.Z * 2, ldb = (uint32_t)x.K * 2;
  Operand oa{gz + (int64_t)s.row * lda, lda, (uint32_t)s.rows * lda};
  Operand ob{w + (int64_t)s.e * x.Z * ldb + n0 * 2, ldb, (uint32_t)n0 * 2};
  P p;
  p.clear();
  p.run(oa, ob, x.Z, s.rows, 0, lds);

  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int m0 = wave / P::WN * P::TM + (lane & 15);
  const int c0 = n0 + wave % P::WN * P::TN + (lane >> 4) * 4;
#pragma unroll
  for (int i = 0; i < P::MI; ++i) {
    const int m = m0 + i * 16;
    if (m >= s.rows) continue;
#pragma unroll
    for (int j = 0; j < P::NJ; ++j) {
      const int col = c0 + j * 16;
      if (col >= x.K) continue;
      const f32x4 v = p.acc[i][j];
      *reinterpret_cast<u32x2*>(gx + (int64_t)(s.row + m) * x.K + col) =
          u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
  }
}

// ---- wgrad: gw[e] = gz^T x

template <typename P, bool F32>
__global__ __launch_bounds__(P::kThreads, 2) void expert_wgrad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ gz,
    const char* __restrict__ a, void* __restrict__ gw, TileGrid<P::BM, P::BN> grid, int64_t base) {
  __shared__ __align__(1024) char lds[P::kLds];
  const Tile tile = grid.at(base + blockIdx.x);
  if (!tile.live) return;
  const int e = tile.grid, z0 = tile.m * P::BM, n0 = tile.n * P::BN;
  const int o0 = x.rows > 0 ? off[e] : 0, rows = x.rows > 0 ? off[e + 1] - o0 : 0;
  const uint32_t lda = (uint32_t)x.Z * 2, ldb = (uint32_t)x.K * 2;
  Operand oa{gz + (int64_t)o0 * lda + z0 * 2, lda, (uint32_t)z0 * 2};
  Operand ob{a + (int64_t)o0 * ldb + n0 * 2, ldb, (uint32_t)n0 * 2};
  P p;
  p.clear();
  p.run(oa, ob, rows, x.Z - z0, 0, lds);

  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int m0 = z0 + wave / P::WN * P::TM + (lane & 15);
  const int c0 = n0 + wave % P::WN * P::TN + (lane >> 4) * 4;
#pragma unroll
  for (int i = 0; i < P::MI; ++i) {
    const int m = m0 + i * 16;
    if (m >= x.Z) continue;
#pragma unroll
    for (int j = 0; j < P::NJ; ++j) {
      const int col = c0 + j * 16;
      if (col >= x.K) continue;
      const f32x4 v = p.acc[i][j];
      const int64_t at = ((int64_t)e * x.Z + m) * x.K + col;
      if constexpr (F32)
        *reinterpret_cast<f32x4*>(static_cast<float*>(gw) + at) = v;
      else
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(gw) + at) =
            u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
  }
}

// ---- the activation's gradient, and the bias gradient

constexpr int kActCols = 32;  // 16-byte chunks of a row a block
constexpr int kActRows = 8;   // rows at a time

// One block per slot of kBiasRows rows and strip of 256 columns of grad_y.  A
// thread owns 8 columns and every 8th row; the column sums of the block are
// added in a fixed order.
__global__ __launch_bounds__(kActCols * kActRows) void expert_act_grad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const uint16_t* __restrict__ gy,
    const uint16_t* __restrict__ pre, uint16_t* __restrict__ gz, float* __restrict__ partial,
    int64_t base, int64_t total, int strips) {
  __shared__ float s_sum[kActRows][kActCols * 8];
  const int64_t tile = base + blockIdx.x;
  if (tile >= total) return;
  const int slot = (int)(tile / strips);
  const Segment s = find_segment(off, x.E, slot, kBiasRows);
  if (s.rows <= 0) return;
  const int c = threadIdx.x % kActCols, r0 = threadIdx.x / kActCols;
  const int col0 = (int)(tile % strips) * (kActCols * 8);
  const int col = col0 + c * 8;
  const bool two = x.Z > x.N;
  float sum[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[h][q] = 0.0f;
  if (col < x.N) {
    for (int r = r0; r < s.rows; r += kActRows) {
      const int64_t row = s.row + r;
      float g[8], z[8], o[8];
      unpack8(*reinterpret_cast<const u32x4*>(gy + row * x.N + col), g);
      if (x.act == MOE_ACT_NONE) {
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = g[q];
      } else {
        unpack8(*reinterpret_cast<const u32x4*>(pre + row * x.Z + col), z);
        float value[8], slope[8];
        act_slopes(x.act, z, value, slope);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = g[q] * slope[q];
        if (two) {
          float up[8], u[8];
          unpack8(*reinterpret_cast<const u32x4*>(pre + row * x.Z + x.N + col), up);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            o[q] *= up[q];
            u[q] = g[q] * value[q];
            sum[1][q] += u[q];
          }
          if (gz != nullptr) *reinterpret_cast<u32x4*>(gz + row * x.Z + x.N + col) = pack8(u);
        }
        if (gz != nullptr) *reinterpret_cast<u32x4*>(gz + row * x.Z + col) = pack8(o);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[0][q] += o[q];
    }
  }
  if (partial == nullptr) return;
  for (int h = 0; h < (two ? 2 : 1); ++h) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) s_sum[r0][c * 8 + q] = h ? sum[1][q] : sum[0][q];
    __syncthreads();
    const int n = threadIdx.x;  // one column a thread
    float t = 0.0f;
    for (int r = 0; r < kActRows; ++r) t += s_sum[r][n];
    if (col0 + n < x.N) partial[(int64_t)slot * x.Z + h * x.N + col0 + n] = t;
  }
}

__global__ __launch_bounds__(256) void expert_bias_sum_kernel(ExpertDims x,
                                                              const int32_t* __restrict__ off,
                                                              const float* __restrict__ partial,
                                                              float* __restrict__ gb) {
  const int strips = (x.Z + 255) / 256;
  const int e = blockIdx.x / strips, n = blockIdx.x % strips * 256 + threadIdx.x;
  if (n >= x.Z) return;
  const int o0 = x.rows > 0 ? off[e] : 0, rows = x.rows > 0 ? off[e + 1] - o0 : 0;
  const int64_t first = o0 / kBiasRows + e;
  const int used = (rows + kBiasRows - 1) / kBiasRows;
  float t = 0.0f;
  for (int i = 0; i < used; ++i) t += partial[(first + i) * x.Z + n];
  gb[(int64_t)e * x.Z + n] = t;
}

// Launches `total` blocks in ranges of at most kMaxTileBlocks (a multiple of
// the XCDs, so that a block keeps its XCD).
template <typename F>
hipError_t in_ranges(int64_t total, F f) {
  hipError_t e = hipSuccess;
  for (int64_t b = 0; b < total && e == hipSuccess; b += kMaxTileBlocks)
    e = f(dim3((uint32_t)std::min(total - b, kMaxTileBlocks)), b);
  return e;
}

constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <bool GATED>
using RowsTile = TileProduct<256, 256, 2, 4, false, false, GATED>;
using RowsGradTile = TileProduct<128, 256, 1, 4, false, true, false>;
using WgradTile = TileProduct<256, 256, 2, 4, true, true, false>;

}  // namespace

hipError_t launch_expert_rows(const ExpertDims& x, const int32_t* off, const uint16_t* a,
                              const uint16_t* w, const float* bias, const uint16_t* residual,
                              uint16_t* y, uint16_t* pre, hipStream_t s) {
  auto go = [&](auto tile) {
    using P = decltype(tile);
    const TileGrid<P::BM, P::BN> grid(1, x.rows / P::BM + x.E, ceil_div(x.N, P::GATED ? P::BN / 2 : P::BN));
    return in_ranges(grid.blocks(), [&](dim3 blocks, int64_t b) {
      return launch(MOE_KERNEL_EXPERT_ROWS, expert_rows_kernel<P>, blocks, dim3(P::kThreads), 0, s, x,
                    off, reinterpret_cast<const char*>(a), reinterpret_cast<const char*>(w), bias,
                    residual, y, pre, grid, b);
    });
  };
  if (gated(x.act)) return go(RowsTile<true>());
  return go(RowsTile<false>());
}

hipError_t launch_expert_rows_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                                   const uint16_t* w, uint16_t* gx, hipStream_t s) {
  using P = RowsGradTile;
  const TileGrid<P::BM, P::BN> grid(1, x.rows / P::BM + x.E, ceil_div(x.K, P::BN));
  return in_ranges(grid.blocks(), [&](dim3 blocks, int64_t b) {
    return launch(MOE_KERNEL_EXPERT_ROWS_GRAD, expert_rows_grad_kernel<P>, blocks, dim3(P::kThreads), 0,
                  s, x, off, reinterpret_cast<const char*>(gz), reinterpret_cast<const char*>(w), gx,
                  grid, b);
  });
}

hipError_t launch_expert_wgrad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                               const uint16_t* a, void* gw, bool f32, hipStream_t s) {
  using P = WgradTile;
  const TileGrid<P::BM, P::BN> grid(x.E, ceil_div(x.Z, P::BM), ceil_div(x.K, P::BN));
  return in_ranges(grid.blocks(), [&](dim3 blocks, int64_t b) {
    return launch(MOE_KERNEL_EXPERT_WGRAD, f32 ? expert_wgrad_kernel<P, true> : expert_wgrad_kernel<P, false>,
                  blocks, dim3(P::kThreads), 0, s, x, off, reinterpret_cast<const char*>(gz),
                  reinterpret_cast<const char*>(a), gw, grid, b);
  });
}

hipError_t launch_expert_act_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gy,
                                  const uint16_t* pre, uint16_t* gz, float* partial,
                                  hipStream_t s) {
  const int strips = ceil_div(x.N, kActCols * 8);
  const int64_t total = bias_slots(x) * strips;
  return in_ranges(total, [&](dim3 grid, int64_t b) {
    return launch(MOE_KERNEL_EXPERT_ACT_GRAD, expert_act_grad_kernel, grid,
                  dim3(kActCols * kActRows), 0, s, x, off, gy, pre, gz, partial, b, total, strips);
  });
}

hipError_t launch_expert_bias_sum(const ExpertDims& x, const int32_t* off, const float* partial,
                                  float* gb, hipStream_t s) {
  return launch(MOE_KERNEL_EXPERT_BIAS_SUM, expert_bias_sum_kernel,
                dim3((uint32_t)(x.E * ceil_div(x.Z, 256))), dim3(256), 0, s, x, off, partial, gb);
}

}  // namespace moe
