// The experts' matrix products on gfx950, forward and backward: for every
// expert e with receive rows [off[e], off[e + 1])
//   rows       z = x w[e]^T (+ bias, activation, residual)  contracts over K
//   rows grad  gx = gz w[e]                                 contracts over Z
//   wgrad      gw[e] = gz^T x                               contracts over e's rows
//
// A block computes BM x BN tiles, one after another, with bf16 matrix
// instructions (16x16x32) and float32 accumulators that stay in registers.
// Per step of 32 along the contraction both operands' tiles are loaded
// straight into LDS (buffer loads with an LDS destination), three stages deep,
// and a step's fragments are read from LDS while the previous step's are
// multiplied; the loads run on from one tile to the next.
//
// What bounds it.  Products of large square matrices: 8192^3 takes 870 to 940
// us in all three directions (1.17 to 1.27 PFLOP/s, matrix cores busy 65% of
// the cycles at 1.9 GHz; the library's product of the same matrices 777 us, 87%
// at 1.6 GHz).  The experts' products take about the time of their operations
// and that of their bytes, one after the other: 64 experts, 4096 tokens, top-8,
// 2048 -> 2 x 1024 takes 335 to 370 us, where one matrix of the same 275 GFLOP
// takes 250 and the 0.87 GB that it has to read and write 180 at the rate of a
// copy.  Matrix cores are busy in 42% of its cycles (a Zipf batch 34%, both
// gradients in one launch 43%) at 1.75 to 1.93 GHz, so it is memory time that is
// not hidden, not power, that binds them: a CU holds one block (100 KiB of LDS),
// no product runs while its waves load the residual and store y and pre, and the
// operands come twice through L2 (1.3 GB read where 0.67 are needed).  Steps:
// fragments read a step ahead of their products and reads that do not wait
// for loads under way (8192^3 from 1220, 1159 and 1447 us to 883, 870 and
// 877), tiles grouped by XCD (half of that: from 50% of L2 requests missing),
// three short stages instead of two long ones, 64-byte stores, and blocks
// that go on from tile to tile (Zipf batch: 908 to 820 us).  Deeper
// pipelines (four stages), smaller tiles, raised wave priority around the
// products, streaming stores and heavy and light experts interleaved
// measured equal or worse.
//
// An operand whose memory is contiguous along the contraction (x and w of
// `rows`, gz of `rows grad`) is kept in LDS as rows of 32 values (64 bytes),
// one 16-byte read per lane and fragment; an operand that is contiguous across
// it (w of `rows grad`, both of wgrad) as 32 rows along the contraction, read
// through the transposing LDS read.  Both layouts are swizzled so that the
// lanes of a read fall into different banks (no conflict is counted); since a
// load to LDS writes lanes one after another, the swizzle permutes which
// global chunk a lane loads.
//
// Rows of different experts never share a tile.  The counts are only known
// on the device: every block builds the list of the experts' row tiles in LDS
// (about 2 us) and finds a tile's expert by searching it.
//
// Loads go through buffer descriptors that end with the operand's rows, so
// rows past the end read as zeros; columns past the width of a transposed
// operand give results that are not stored.  Chunks past the end of a
// contiguous contraction are sent past the descriptor's end, so that they
// read as zeros on both sides (0 * NaN would not be 0).
#include <algorithm>
#include <type_traits>

#include "block_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
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

__device__ __forceinline__ u32x4 pack_two(f32x4 lo, f32x4 hi) {
  return u32x4{bf16_pair(lo[0], lo[1]), bf16_pair(lo[2], lo[3]), bf16_pair(hi[0], hi[1]),
               bf16_pair(hi[2], hi[3])};
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

// The normal distribution Phi(z), and bell = exp(-z^2 / 2).  With x = |z| / sqrt 2,
// erfc(x) = bell * t * P(t), t = 1 / (1 + 0.425 x): P is a polynomial of degree
// 7, fitted (iteratively reweighted least squares at Chebyshev nodes) so that
// t * P(t) has a relative error below 2.2e-7 over |z| < 15.  In float32 the
// tail's relative error stays below (z^2 + 32) 2^-24, the share of z^2 from the
// argument of exp; over every bf16 z it measured 5e-7 for |z| < 1 and 3.4e-6 at
// most, at -12.25.  Beyond -12.9 Phi is below the smallest normal float and may
// be 0.
// A seventh of the instructions of the math library's erfc, which dominated
// the epilogue of small products.
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  bell = __expf(-0.5f * z * z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.425f * 0.70710678118654752f, fabsf(z), 1.0f));
  float p = 0.07013754546642303f;
  p = __builtin_fmaf(p, t, -0.30760806798934937f);
  p = __builtin_fmaf(p, t, 0.39813491702079773f);
  p = __builtin_fmaf(p, t, -0.0946105495095253f);
  p = __builtin_fmaf(p, t, 0.25057145953178406f);
  p = __builtin_fmaf(p, t, 0.2020537555217743f);
  p = __builtin_fmaf(p, t, 0.24162858724594116f);
  p = __builtin_fmaf(p, t, 0.23969215154647827f);
  const float tail = 0.5f * bell * t * p;
  return z < 0.0f ? tail : 1.0f - tail;
}

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
      for (int q = 0; q < 8; ++q) {
        float bell;
        z[q] *= normal_cdf(z[q], bell);
      }
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
        float bell;
        const float p = normal_cdf(z[q], bell);
        value[q] = z[q] * p;
        slope[q] = p + z[q] * 0.3989422804014327f * bell;
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

// ---- which expert and rows a tile of rows stands for

// The experts' row tiles, numbered without gaps: expert e's are
// [first[e], first[e + 1]).  Built in LDS by every block.
struct RowTiles {
  int32_t first[MOE_MAX_EXPERTS + 1];
  int32_t wave[16];

  // BM rows a tile; THREADS threads, all of the block.
  template <int BM, int THREADS>
  __device__ __forceinline__ void build(const int32_t* off, int E) {
    constexpr int per = MOE_MAX_EXPERTS / THREADS;  // consecutive experts a thread
    static_assert(per * THREADS == MOE_MAX_EXPERTS && THREADS / kWave <= 16);
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
    int n[per], sum = 0;
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int e = tid * per + q;
      n[q] = e < E ? (off[e + 1] - off[e] + BM - 1) / BM : 0;
      sum += n[q];
    }
    int before = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(before, d);
      if (lane >= d) before += o;
    }
    if (lane == kWave - 1) wave[wv] = before;
    __syncthreads();
    before -= sum;
    for (int q = 0; q < wv; ++q) before += wave[q];
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int e = tid * per + q;
      if (e < E) first[e] = before;
      before += n[q];
      if (e == E - 1) first[E] = before;
    }
    __syncthreads();
  }
};

struct Segment {
  int e;     // expert
  int row;   // first row
  int rows;  // rows of the tile
};

// The expert of row tile m: the last one with first[e] <= m.  Two rounds of
// one LDS read a lane: every ceil(E / 64)-th expert, then those in between.
template <int BM>
__device__ __forceinline__ Segment segment_of(const RowTiles& t, const int32_t* off, int E, int m) {
  const int lane = threadIdx.x & (kWave - 1);
  const int step = (E + kWave - 1) / kWave;
  const int e1 = lane * step;
  int e = (__popcll(__ballot(e1 < E && t.first[min(e1, E)] <= m)) - 1) * step;  // lane 0 is in
  if (step > 1) {
    const int e2 = e + lane;
    e += __popcll(__ballot(lane < step && e2 < E && t.first[min(e2, E)] <= m)) - 1;
  }
  Segment s;
  s.e = __builtin_amdgcn_readfirstlane(e);
  s.row = off[s.e] + (m - __builtin_amdgcn_readfirstlane(t.first[s.e])) * BM;
  s.rows = min(BM, off[s.e + 1] - s.row);
  return s;
}

// The same for slots of bm rows that need no table: expert e's slots start at
// off[e] / bm + e, which leaves at least ceil(rows / bm) slots each and makes
// rows / bm + E in all; slots that no row falls into have rows <= 0.
__device__ __forceinline__ Segment segment_of_slot(const int32_t* off, int E, int slot, int bm) {
  const int lane = threadIdx.x & (kWave - 1);
  const int step = (E + kWave - 1) / kWave;
  const int e1 = lane * step;
  int e = (__popcll(__ballot(e1 < E && off[min(e1, E)] / bm + e1 <= slot)) - 1) * step;
  if (step > 1) {
    const int e2 = e + lane;
    e += __popcll(__ballot(lane < step && e2 < E && off[min(e2, E)] / bm + e2 <= slot)) - 1;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  Segment s;
  const int o0 = off[e], o1 = off[e + 1];
  s.e = e;
  s.row = o0 + (slot - (o0 / bm + e)) * bm;
  s.rows = min(o1 - s.row, bm);
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

  __host__ __device__ TileGrid(int grids_, int mtiles_, int ntiles_)
      : grids(grids_), mtiles(mtiles_), ntiles(ntiles_),
        mgroups((mtiles_ + kGroupM - 1) / kGroupM), ngroups((ntiles_ + kGroupN - 1) / kGroupN) {}
  // Numbers at() takes: those of tiles, and some that are not live.
  __host__ __device__ int numbers() const {
    return (grids * mgroups * ngroups + kXcds - 1) / kXcds * kXcds * kTiles;
  }
  __device__ __forceinline__ Tile at(int number) const {
    const int i = number / kXcds;
    const int group = i / kTiles * kXcds + number % kXcds;
    const int in = i % kTiles;
    const int per = mgroups * ngroups;
    const int g = group % per;
    Tile t;
    t.live = group / per < grids;
    t.grid = group / per;
    t.m = g / ngroups * kGroupM + in / kGroupN;
    t.n = g % ngroups * kGroupN + in % kGroupN;
    t.live = t.live && t.m < mtiles && t.n < ntiles;
    return t;
  }
};

// ---- the tile product

template <int BM_, int BN_, int WM_, int WN_, bool AT_, bool BT_, bool GATED_>
struct TileProduct {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr bool AT = AT_, BT = BT_, GATED = GATED_;
  static constexpr int kNW = WM * WN, kThreads = kNW * kWave;
  // A wave computes every WM-th 16 rows (MI of them) and TN consecutive columns.
  static constexpr int TN = BN / WN, MI = BM / WM / 16, NJ = TN / 16;
  static constexpr int kABytes = BM * kBK * 2, kBBytes = BN * kBK * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 3;
  static constexpr int kLds = kStages * kStage;
  static constexpr int QA = kABytes / 1024 / kNW, QB = kBBytes / 1024 / kNW;  // loads a wave and stage
  static_assert(QA * kNW * 1024 == kABytes && QB * kNW * 1024 == kBBytes);
  static_assert(TN == 64, "the order of a wave's columns is of 64");

  // Columns of B.  A lane gets four consecutive result columns of each of a
  // wave's four fragments; lane group g (of four) is given columns
  // 32 (j / 2) + 8 g + 4 (j % 2) + 0..3 of the wave's 64 for fragment j, so that two
  // fragments make 16 bytes of bf16 and the four groups 64 consecutive bytes
  // of a result row.  (Stores that cover less of a line cost the most where
  // results outweigh operands: with 32 bytes a row and the streaming hint,
  // which keeps L2 from joining them, the weight gradient of a Zipf batch took
  // 1250 us instead of 830.)
  //
  // Contiguous contraction: LDS row r (64 bytes, 4 chunks) holds chunk
  // p ^ swizzle(r) at position p.  A's rows are read in order, B's in the order
  // above (rows i % 4 + 8 (i / 4) for lane i); each has the swizzle that spreads
  // its own eight consecutive lanes over all banks.
  template <bool B>
  static __device__ __forceinline__ int swizzle(int r) {
    return B ? ((r >> 1) & 1) | ((r >> 3) & 1) << 1 : (r >> 1) & 3;
  }
  // Transposed: LDS row kr (along the contraction) holds W columns in units of
  // 16 bytes; unit u is at position u ^ spread(kr).
  static __device__ __forceinline__ int spread(int kr) {
    return (kr & 3) << 2 | ((kr >> 3) & 1) << 1;
  }
  // Byte offset in memory of a lane's 16 bytes for the wave's q-th load.
  template <int W>
  static __device__ __forceinline__ uint32_t offset_t(uint32_t ld, int wave, int lane, int q) {
    constexpr int per = W / 8;       // units a row
    const int pos = (q * kNW + wave) * 64 + lane;
    const int kr = pos / per, p = pos % per;
    return kr * ld + (p ^ spread(kr)) * 16;
  }

  // Memory row of B's LDS row r.  Gated: a wave's first 32 rows are of the
  // gate, the other 32 the same columns of the up projection.
  static __device__ __forceinline__ int b_row(int r, int gate_up) {
    if constexpr (!GATED) return r;
    return r / 64 * 32 + (r & 31) + ((r >> 5) & 1) * gate_up;
  }

  struct Fragments {
    bf16x8 a[MI], b[NJ];
  };

  // A tile's operands, as far as they have been loaded.
  struct Cursor {
    const char *a, *b;         // row 0, contraction 0 of the tile
    uint32_t a_bytes, b_bytes; // contiguous contraction: bytes to the end of the tile's rows;
                               // transposed: bytes from a memory row's start to the tile's columns
    int len;                   // contraction elements
    int step;                  // step that is loaded next
  };
  // Steps of a tile: an even number, for the two sets of fragment registers,
  // and at least four, so that the loads are never more than a tile ahead.
  static __device__ __forceinline__ int steps_of(int len) {
    return max((len + 2 * kBK - 1) / (2 * kBK), 2) * 2;
  }

  f32x4 acc[MI][NJ];
  uint32_t va[QA], vb[QB];  // byte offsets of this lane's loads from a step's base
  uint32_t lda, ldb;        // bytes between memory rows
  char* lds;
  int wave, lane, m0, n0;
  int put;                  // LDS offset of the stage to load next

  // gate_up: memory rows from the gate's to the up projection's row (gated only).
  __device__ __forceinline__ TileProduct(char* lds_, uint32_t lda_, uint32_t ldb_, int gate_up)
      : lda(lda_), ldb(ldb_), lds(lds_), put(0) {
    lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    m0 = wave / WN * 16;
    n0 = wave % WN * TN;
#pragma unroll
    for (int q = 0; q < QA; ++q)
      va[q] = AT ? offset_t<BM>(lda, wave, lane, q)
                 : (uint32_t)row_of(q) * lda + chunk<false>() * 16;
#pragma unroll
    for (int q = 0; q < QB; ++q)
      vb[q] = BT ? offset_t<BN>(ldb, wave, lane, q)
                 : (uint32_t)b_row(row_of(q), gate_up) * ldb + chunk<true>() * 16;
  }

  // Contiguous contraction: the LDS row of this lane's q-th load, and the chunk
  // of a step that it loads (the same for every q).
  __device__ __forceinline__ int row_of(int q) const { return (q * kNW + wave) * 16 + lane / 4; }
  template <bool B>
  __device__ __forceinline__ int chunk() const {
    static_assert(kNW % 2 == 0);
    return (lane & 3) ^ swizzle<B>(row_of(0));
  }

  // Loads the cursor's step into the stage at `to`.
  __device__ __forceinline__ void load(Cursor& c, char* to) {
    const int done = c.step * kBK, left = c.len - done;
    issue<AT, false, QA>(c.a, lda, c.a_bytes, va, done, left, to + wave * 1024);
    issue<BT, true, QB>(c.b, ldb, c.b_bytes, vb, done, left, to + kABytes + wave * 1024);
    ++c.step;
  }

  static __device__ __forceinline__ int stage_after(int at) {
    return at == (kStages - 1) * kStage ? 0 : at + kStage;
  }

  // Loads the first tile's first three steps.
  __device__ __forceinline__ void start(Cursor& c) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) load(c, lds + i * kStage);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // acc = A B of one tile of `steps` steps (acc += A B without `clear`).  rows:
  // result rows that are wanted
  // (the others' products are skipped, a quarter of the tile at a time).
  // next(cursor) sets the cursor to the following tile (or to an empty one).
  //
  // While the fragments of step s (in registers) are multiplied, those of
  // step s + 1 are read from LDS and the loads of steps s + 2 and s + 3 are
  // under way; steps past the end are the next tile's, so the loads never
  // pause and run on under the epilogue.  One barrier a step: before it a
  // wave waits for its own fragments of step s (so stage s is free after it,
  // for step s + 3) and for its own loads of step s + 1 (so they can be read
  // after it).  Loads come back in the order they were issued, so with at most
  // one step's count of operations under way, those are the last step's.
  template <typename Next>
  __device__ __forceinline__ void run(Cursor& c, const Next& next, int steps, int rows,
                                      bool clear = true) {
    if (clear) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    Fragments f0, f1;
    wait_and_meet<-1>();  // the tile's first three steps have landed, for every wave
    read(f0, lds + put);
    for (int s = 0; s < steps; s += 2) {
      step(c, s == 0, rows, f0, f1);
      // Tiles have an even number of steps and the cursor is three or four
      // ahead here, so it comes to a tile's end in this place.
      if (c.step == steps) next(c);
      step(c, s == 0, rows, f1, f0);
    }
    // What is under way has landed before the epilogue's stores are issued, so
    // the next tile's first steps need not wait for those.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // One step.  landed: what it reads has landed.  (The last step of a tile
  // reads the next tile's first fragments, which that tile reads again.)
  __device__ __forceinline__ void step(Cursor& c, bool landed, int rows, const Fragments& now,
                                       Fragments& then) {
    if (landed)
      wait_and_meet<-1>();
    else
      wait_and_meet<QA + QB>();
    refill(c, then, lds + put, lds + stage_after(put));
    put = stage_after(put);
    multiply<0>(now);
    interleave();
    __builtin_amdgcn_sched_barrier(0);
    if (rows > kQuarter) multiply<1>(now);
    __builtin_amdgcn_sched_barrier(0);
    if (rows > 2 * kQuarter) multiply<2>(now);
    __builtin_amdgcn_sched_barrier(0);
    if (rows > 3 * kQuarter) multiply<3>(now);
    __builtin_amdgcn_sched_barrier(0);
  }

  // Quarter Q of the tile's rows.
  static constexpr int kQuarter = BM / 4;
  template <int Q>
  __device__ __forceinline__ void multiply(const Fragments& f) {
#pragma unroll
    for (int i = Q * MI / 4; i < (Q + 1) * MI / 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
  }

  // Asks the scheduler to start with products (whose fragments have been
  // waited for) and to spread the loads and the reads between them.
  static __device__ __forceinline__ void interleave() {
    constexpr int loads = QA + QB, reads = MI * (AT ? 2 : 1) + NJ * (BT ? 2 : 1);
    constexpr int products = MI * NJ / 4;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instructions
#pragma unroll
    for (int i = 1; i < products; ++i) {
      constexpr int each = (reads + products - 2) / (products - 1);
      __builtin_amdgcn_sched_group_barrier(0x100, each, 0);  // LDS reads
      if (i <= loads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // load
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  }

  __device__ __forceinline__ void read(Fragments& f, const char* from) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) f.b[j] = fragment<BT, true, BN>(from + kABytes, n0, j, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i) f.a[i] = fragment<AT, false, BM>(from, m0, i * WM, lane);
  }

  // The loads of a later step and the reads of the next.  The two stages are
  // different ones, and saying so (restrict) matters: where the compiler sees
  // that a read from LDS may touch what a load to LDS writes, it waits for
  // every load under way before the read.
  __device__ __forceinline__ void refill(Cursor& c, Fragments& f, char* __restrict__ to,
                                         const char* __restrict__ from) {
    load(c, to);
    read(f, from);
  }

  // Waits until none of this wave's LDS reads and at most N (< 0: any number)
  // of its loads are under way, then for the block's other waves.
  template <int N>
  static __device__ __forceinline__ void wait_and_meet() {
    if constexpr (N < 0)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  template <bool T, bool B, int Q>
  __device__ __forceinline__ void issue(const char* from, uint32_t ld, uint32_t limit,
                                        const uint32_t (&v)[Q], int done, int left, char* at) const {
    const char* base;
    uint32_t bytes;
    if constexpr (T) {
      base = from + (int64_t)done * ld;
      bytes = (uint32_t)max(min(left, kBK), 0) * ld;
      bytes = bytes > limit ? bytes - limit : 0;
    } else {
      base = from + (int64_t)done * 2;
      bytes = left > 0 && limit > (uint32_t)done * 2 ? limit - done * 2 : 0;
    }
    const __amdgpu_buffer_rsrc_t r = uniform_buffer(base, bytes);
    const bool in = T || chunk<B>() * 8 < left;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void*)(at + q * kNW * 1024), 16,
                                               in ? v[q] : kPast, 0, 0, 0);
  }

  // This lane's part of fragment f of an operand whose wave starts at `first`.
  template <bool T, bool B, int W>
  static __device__ __forceinline__ bf16x8 fragment(const char* tile, int first, int f, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (T) {
      // Lane i names 4 columns (8 bytes) of row i / 4 and gets column i of four rows.
      const int kr = g * 8 + (i >> 2), piece = i & 3;
      const int col = first + (B ? f / 2 * 32 + piece * 8 + f % 2 * 4 : f * 16 + piece * 4);
      const char* p = tile + kr * (W * 2) + (((col >> 3) ^ spread(kr)) << 4) + (col & 4) * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(p + 4 * W * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = first + (B ? f / 2 * 32 + (i >> 2) * 8 + f % 2 * 4 + (i & 3) : f * 16 + i);
      const char* p = tile + r * 64 + ((g ^ swizzle<B>(r)) << 4);
      return *reinterpret_cast<const bf16x8*>(p);
    }
  }
};

// A lane of acc[i][j] holds four results of row m0 + i * WM * 16 + lane % 16 of
// the tile, in the columns described above.

// Blocks of a launch: each CU gets as many as fit its LDS, and every block
// computes one tile after another (numbers blockIdx.x, + gridDim.x, ...).
constexpr int kCus = 256;
template <typename P>
constexpr int blocks_at_once() {
  return kCus * (P::kLds + (int)sizeof(RowTiles) <= 80 * 1024 ? 2 : 1);
}

// ---- rows: y = act(x w^T + bias) + residual

// The epilogue of four of a lane's rows (of the wave's 16 * MI), columns c0 on:
// i0.. are the accumulator's rows.
template <typename P, int I0>
__device__ __forceinline__ void rows_epilogue(const P& p, const ExpertDims& x, const Segment& s,
                                              int c0, const float (&bz)[16],
                                              const uint16_t* residual, uint16_t* y,
                                              uint16_t* pre) {
  constexpr int kRows = 4, kHalves = P::GATED ? 1 : 2;  // rows, and 8-column pieces of y in a row
  int64_t row[kRows];
  bool ok[kRows];
  u32x4 res[kRows][kHalves];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int m = p.m0 + (I0 + i) * (P::WM * 16) + (p.lane & 15);
    ok[i] = m < s.rows;
    row[i] = s.row + (ok[i] ? m : 0);
  }
  if (residual != nullptr) {  // all loads before the first use
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        res[i][h] = *reinterpret_cast<const u32x4*>(residual + row[i] * x.N +
                                                    (c0 + h * 32 < x.N ? c0 + h * 32 : 0));
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float z[2][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = j * 4 + q;
        z[n / 8][n % 8] = p.acc[I0 + i][j][q] + bz[n];
      }
    if (!ok[i]) continue;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int col = c0 + h * 32;
      if (col >= x.N) continue;
      float out[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] = z[h][q];
      if (pre != nullptr) {
        *reinterpret_cast<u32x4*>(pre + row[i] * x.Z + col) = pack8(z[h]);
        if constexpr (P::GATED)
          *reinterpret_cast<u32x4*>(pre + row[i] * x.Z + x.N + col) = pack8(z[1]);
      }
      act_values(x.act, out);
      if constexpr (P::GATED) {
#pragma unroll
        for (int q = 0; q < 8; ++q) out[q] *= z[1][q];
      }
      if (residual != nullptr) {
        float r[8];
        unpack8(res[i][h], r);
#pragma unroll
        for (int q = 0; q < 8; ++q) out[q] += r[q];
      }
      *reinterpret_cast<u32x4*>(y + row[i] * x.N + col) = pack8(out);
    }
  }
}

template <typename P>
__global__ __launch_bounds__(P::kThreads, 2) void expert_rows_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ a,
    const char* __restrict__ w, const float* __restrict__ bias,
    const uint16_t* __restrict__ residual, uint16_t* __restrict__ y, uint16_t* __restrict__ pre,
    int ntiles) {
  __shared__ __align__(1024) char lds[P::kLds + sizeof(RowTiles)];
  RowTiles& table = *reinterpret_cast<RowTiles*>(lds + P::kLds);
  constexpr int kCols = P::GATED ? P::BN / 2 : P::BN;  // columns of y a tile
  table.build<P::BM, P::kThreads>(off, x.E);
  const TileGrid<P::BM, P::BN> grid(1, __builtin_amdgcn_readfirstlane(table.first[x.E]), ntiles);
  const int numbers = grid.numbers();
  const uint32_t ld = (uint32_t)x.K * 2;
  // The tile that is loaded, at most one ahead of the one that is multiplied.
  int number = blockIdx.x, n_ahead = 0;
  Segment ahead{0, 0, 0};
  auto next = [&](typename P::Cursor& c) {
    c = {a, w, 0, 0, 0, 0};  // no tile left: loads nothing
    ahead.rows = 0;
    for (; number < numbers; number += gridDim.x) {
      const Tile t = grid.at(number);
      if (!t.live) continue;
      const Segment s = ahead = segment_of<P::BM>(table, off, x.E, t.m);
      const int n0 = n_ahead = t.n * kCols;
      c.a = a + (int64_t)s.row * ld;
      c.a_bytes = (uint32_t)s.rows * ld;
      c.b = w + ((int64_t)s.e * x.Z + n0) * ld;
      c.b_bytes = (uint32_t)(x.Z - n0) * ld;
      c.len = x.K;
      number += gridDim.x;
      break;
    }
  };
  typename P::Cursor c;
  next(c);
  P p(lds, ld, ld, x.N);
  p.start(c);
  while (ahead.rows > 0) {
    const Segment s = ahead;
    const int col0 = n_ahead;
    p.run(c, next, P::steps_of(x.K), s.rows);

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
    static_assert(P::MI % 4 == 0 && P::MI <= 8);
    rows_epilogue<P, 0>(p, x, s, c0, bz, residual, y, pre);
    if constexpr (P::MI > 4) rows_epilogue<P, 4>(p, x, s, c0, bz, residual, y, pre);
  }
}

// ---- rows of few tokens: the same product where an expert has a few rows

// Decoding: every used expert's weights are read once for a handful of rows,
// so the product is bound by that read and needs many loads under way rather
// than tiles.  One block computes 16 columns of y (of gate and up, when gated)
// for one expert; its waves split the contraction, read weights and rows
// straight into matrix-instruction registers, kFewSteps steps (32 values each)
// at a time, and add their parts through LDS in a fixed order.  MT * 16 rows a
// pass; an expert with more takes further passes, which find the weights in L2.
// 16 tokens, top-8 of 64 experts, 2048 -> 2 x 1024 (474 MB, nearly all weights): 86 us,
// 5.5 TB/s, where tiles take 113; one token (67 MB) 13.3 us, 5.0 TB/s.
constexpr int kFewWaves = 4;
constexpr int kFewSteps = 8;

template <int MT, bool GATED>
__global__ __launch_bounds__(kFewWaves * kWave) void expert_few_rows_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ a,
    const char* __restrict__ w, const float* __restrict__ bias,
    const uint16_t* __restrict__ residual, uint16_t* __restrict__ y, uint16_t* __restrict__ pre,
    int strips, int64_t base) {
  constexpr int H = GATED ? 2 : 1;
  __shared__ float part[kFewWaves][MT * H][256];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t block = base + blockIdx.x;
  const int which = (int)(block / strips), col0 = (int)(block % strips) * 16;
  int e = which;
  if (x.rows < x.E) {
    // Fewer rows than experts: `which` is a row (of the band), and the block of
    // its expert's first row does the work.
    const int row = off[0] + which;
    const int step = (x.E + kWave - 1) / kWave;
    const int e1 = lane * step;
    e = (__popcll(__ballot(e1 < x.E && off[min(e1, x.E)] <= row)) - 1) * step;
    if (step > 1) {
      const int e2 = e + lane;
      e += __popcll(__ballot(lane < step && e2 < x.E && off[min(e2, x.E)] <= row)) - 1;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (off[e] != row) return;
  }
  const int o0 = off[e], rows = off[e + 1] - o0;
  const uint32_t ld = (uint32_t)x.K * 2;
  const int steps = (x.K + 31) / 32;
  const int first = wave * steps / kFewWaves, last = (wave + 1) * steps / kFewWaves;
  const int i = lane & 15, g = lane >> 4;
  const __amdgpu_buffer_rsrc_t rw = uniform_buffer(w + (int64_t)e * x.Z * ld, (uint32_t)x.Z * ld);
  // (col0 + i may be past the last column: such rows of w give results that are not stored, or
  // are past the descriptor's end.)
  const uint32_t vw = (uint32_t)(col0 + i) * ld + g * 16, up = (uint32_t)x.N * ld;
  for (int r0 = 0; r0 < rows; r0 += MT * 16) {
    const __amdgpu_buffer_rsrc_t rx = uniform_buffer(
        a + (int64_t)(o0 + r0) * ld, (uint32_t)min(rows - r0, MT * 16) * ld);  // rows past the end: zeros
    f32x4 acc[MT][H];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < H; ++h) acc[m][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = first; s < last; s += kFewSteps) {
      bf16x8 fw[kFewSteps][H], fx[kFewSteps][MT];
#pragma unroll
      for (int q = 0; q < kFewSteps; ++q) {
        // Steps past this wave's part and chunks past the row's end read zeros.
        const bool in = s + q < last && (s + q) * 32 + g * 8 < x.K;
        const uint32_t k = (uint32_t)(s + q) * 64;
#pragma unroll
        for (int h = 0; h < H; ++h)
          fw[q][h] = __builtin_bit_cast(
              bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rw, in ? vw + h * up + k : kPast, 0, 0));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          fx[q][m] = __builtin_bit_cast(
              bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                          rx, in ? (uint32_t)(m * 16 + i) * ld + g * 16 + k : kPast, 0, 0));
      }
#pragma unroll
      for (int q = 0; q < kFewSteps; ++q)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < H; ++h)
            acc[m][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[q][h], fx[q][m], acc[m][h], 0, 0, 0);
    }
    // acc[m][h][q]: column g * 4 + q, row m * 16 + i.
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < H; ++h)
        *reinterpret_cast<f32x4*>(&part[wave][m * H + h][i * 16 + g * 4]) = acc[m][h];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += kFewWaves * kWave) {
      const int m = t / 256, r = r0 + m * 16 + t % 256 / 16, col = col0 + t % 16;
      if (r >= rows || col >= x.N) continue;
      float z[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        z[h] = 0.0f;
#pragma unroll
        for (int q = 0; q < kFewWaves; ++q) z[h] += part[q][m * H + h][t % 256];
        if (bias != nullptr) z[h] += bias[(int64_t)e * x.Z + h * x.N + col];
      }
      const int64_t row = o0 + r;
      float out[8] = {z[0]};
      if (pre != nullptr) {
#pragma unroll
        for (int h = 0; h < H; ++h)
          pre[row * x.Z + h * x.N + col] = (uint16_t)bf16_pair(z[h], 0.0f);
      }
      act_values(x.act, out);
      if constexpr (GATED) out[0] *= z[1];
      if (residual != nullptr)
        out[0] += __uint_as_float((uint32_t)residual[row * x.N + col] << 16);
      y[row * x.N + col] = (uint16_t)bf16_pair(out[0], 0.0f);
    }
    __syncthreads();
  }
}

// ---- rows grad: gx = gz w

// Block `block` of `blocks`; lds: P::kLds + sizeof(RowTiles) bytes.
template <typename P>
__device__ __forceinline__ void rows_grad(const ExpertDims& x, const int32_t* off, const char* gz,
                                          const char* w, uint16_t* gx, int ntiles, char* lds,
                                          int block, int blocks) {
  RowTiles& table = *reinterpret_cast<RowTiles*>(lds + P::kLds);
  table.build<P::BM, P::kThreads>(off, x.E);
  const TileGrid<P::BM, P::BN> grid(1, __builtin_amdgcn_readfirstlane(table.first[x.E]), ntiles);
  const int numbers = grid.numbers();
  const uint32_t lda = (uint32_t)x.Z * 2, ldb = (uint32_t)x.K * 2;
  int number = block, n_ahead = 0;
  Segment ahead{0, 0, 0};
  auto next = [&](typename P::Cursor& c) {
    c = {gz, w, 0, 0, 0, 0};
    ahead.rows = 0;
    for (; number < numbers; number += blocks) {
      const Tile t = grid.at(number);
      if (!t.live) continue;
      const Segment s = ahead = segment_of<P::BM>(table, off, x.E, t.m);
      n_ahead = t.n * P::BN;
      c.a = gz + (int64_t)s.row * lda;
      c.a_bytes = (uint32_t)s.rows * lda;
      c.b = w + (int64_t)s.e * x.Z * ldb + t.n * P::BN * 2;
      c.b_bytes = (uint32_t)(t.n * P::BN * 2);
      c.len = x.Z;
      number += blocks;
      break;
    }
  };
  typename P::Cursor c;
  next(c);
  P p(lds, lda, ldb, 0);
  p.start(c);
  while (ahead.rows > 0) {
    const Segment s = ahead;
    const int col0 = n_ahead;
    p.run(c, next, P::steps_of(x.Z), s.rows);

    const int c0 = col0 + p.n0 + (p.lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < P::MI; ++i) {
      const int m = p.m0 + i * (P::WM * 16) + (p.lane & 15);
      if (m >= s.rows) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = c0 + h * 32;
        if (col >= x.K) continue;
        *reinterpret_cast<u32x4*>(gx + (int64_t)(s.row + m) * x.K + col) =
            pack_two(p.acc[i][2 * h], p.acc[i][2 * h + 1]);
      }
    }
  }
}

// ---- wgrad: gw[e] = gz^T x

// Block `block` of `blocks`; lds: P::kLds bytes.
template <typename P, bool F32>
__device__ __forceinline__ void wgrad(const ExpertDims& x, const int32_t* off, const char* gz,
                                      const char* a, void* gw,
                                      const TileGrid<P::BM, P::BN>& grid, char* lds, int block,
                                      int blocks) {
  const int numbers = grid.numbers();
  const uint32_t lda = (uint32_t)x.Z * 2, ldb = (uint32_t)x.K * 2;
  // A tile's bands follow each other.
  int number = block, band = x.bands - 1;
  Tile ahead{0, 0, 0, false};
  auto next = [&](typename P::Cursor& c) {
    c = {gz, a, 0, 0, 0, 0};
    if (++band < x.bands) number -= blocks;
    band = band < x.bands ? band : 0;
    ahead.live = false;
    for (; number < numbers; number += blocks) {
      const Tile t = grid.at(number);
      if (!t.live) continue;
      ahead = t;
      const int32_t* o = off + (int64_t)band * (x.E + 1) + t.grid;
      const int64_t o0 = x.rows > 0 ? o[0] : 0;
      c.a = gz + o0 * lda + t.m * P::BM * 2;
      c.a_bytes = (uint32_t)(t.m * P::BM * 2);
      c.b = a + o0 * ldb + t.n * P::BN * 2;
      c.b_bytes = (uint32_t)(t.n * P::BN * 2);
      c.len = x.rows > 0 ? o[1] - (int)o0 : 0;
      number += blocks;
      break;
    }
  };
  typename P::Cursor c;
  next(c);
  P p(lds, lda, ldb, 0);
  p.start(c);
  while (ahead.live) {
    const Tile t = ahead;
    const int b = band;
    p.run(c, next, P::steps_of(c.len), x.Z - t.m * P::BM, b == 0);
    if (b + 1 < x.bands) continue;

    const int r0 = t.m * P::BM + p.m0 + (p.lane & 15);
    const int c0 = t.n * P::BN + p.n0 + (p.lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < P::MI; ++i) {
      const int m = r0 + i * (P::WM * 16);
      if (m >= x.Z) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = c0 + h * 32;
        if (col >= x.K) continue;
        const f32x4 lo = p.acc[i][2 * h], hi = p.acc[i][2 * h + 1];
        const int64_t at = ((int64_t)t.grid * x.Z + m) * x.K + col;
        if constexpr (F32) {
          f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(gw) + at);
          o[0] = lo;
          o[1] = hi;
        } else {
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(gw) + at) = pack_two(lo, hi);
        }
      }
    }
  }
}

// grad_bias: the partial sums of an expert's slots, one column a thread (block
// `block` of THREADS columns), eight loads at a time.
template <int THREADS>
__device__ __forceinline__ void bias_sum(const ExpertDims& x, const int32_t* __restrict__ off,
                                         const float* __restrict__ partial, float* __restrict__ gb,
                                         int block) {
  const int strips = (x.Z + THREADS - 1) / THREADS;
  const int e = block / strips, n = block % strips * THREADS + threadIdx.x;
  if (n >= x.Z) return;
  float t = 0.0f;
  for (int b = 0; b < (x.rows > 0 ? x.bands : 0); ++b) {
    const int o0 = off[b * (x.E + 1) + e], rows = off[b * (x.E + 1) + e + 1] - o0;
    const int used = (rows + kBiasRows - 1) / kBiasRows;
    const float* p = partial + (o0 / kBiasRows + e + (int64_t)b * x.E) * x.Z + n;
    int i = 0;
    for (; i + 8 <= used; i += 8, p += (int64_t)8 * x.Z) {  // eight loads at a time, added in order
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = p[(int64_t)q * x.Z];
#pragma unroll
      for (int q = 0; q < 8; ++q) t += v[q];
    }
    for (; i < used; ++i, p += x.Z) t += *p;
  }
  gb[(int64_t)e * x.Z + n] = t;
}

// Bound by the longest chain of loads: 30 experts of 136 rows 4.0 us, which any launch
// takes; one expert of 8192 rows among 64 (256 slots) 19.6.
constexpr int kBiasThreads = 256;
__global__ __launch_bounds__(kBiasThreads) void expert_bias_sum_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const float* __restrict__ partial,
    float* __restrict__ gb) {
  bias_sum<kBiasThreads>(x, off, partial, gb, blockIdx.x);
}

// ---- the kernels of the two gradients, apart and in one launch

template <typename P>
__global__ __launch_bounds__(P::kThreads, 2) void expert_rows_grad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ gz,
    const char* __restrict__ w, uint16_t* __restrict__ gx, int ntiles) {
  __shared__ __align__(1024) char lds[P::kLds + sizeof(RowTiles)];
  rows_grad<P>(x, off, gz, w, gx, ntiles, lds, blockIdx.x, gridDim.x);
}

template <typename P, bool F32>
__global__ __launch_bounds__(P::kThreads, 2) void expert_wgrad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ gz,
    const char* __restrict__ a, void* __restrict__ gw, TileGrid<P::BM, P::BN> grid) {
  __shared__ __align__(1024) char lds[P::kLds];
  wgrad<P, F32>(x, off, gz, a, gw, grid, lds, blockIdx.x, gridDim.x);
}

// The first bias_blocks blocks compute gb, the next row_blocks gx, the others gw.
template <typename PR, typename PW, bool F32>
__global__ __launch_bounds__(PR::kThreads, 2) void expert_grads_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const char* __restrict__ gz,
    const char* __restrict__ w, uint16_t* __restrict__ gx, int ntiles,
    const char* __restrict__ a, void* __restrict__ gw, TileGrid<PW::BM, PW::BN> grid,
    const float* __restrict__ partial, float* __restrict__ gb, int row_blocks, int bias_blocks) {
  static_assert(PR::kThreads == PW::kThreads && PR::kLds >= PW::kLds);
  __shared__ __align__(1024) char lds[PR::kLds + sizeof(RowTiles)];
  const int block = (int)blockIdx.x - bias_blocks;
  if (block < 0)
    bias_sum<PR::kThreads>(x, off, partial, gb, blockIdx.x);
  else if (block < row_blocks)
    rows_grad<PR>(x, off, gz, w, gx, ntiles, lds, block, row_blocks);
  else
    wgrad<PW, F32>(x, off, gz, a, gw, grid, lds, block - row_blocks,
                   (int)gridDim.x - bias_blocks - row_blocks);
}

// ---- the activation's gradient, and the bias gradient

constexpr int kActCols = 32;  // 16-byte chunks of a row a block
constexpr int kActRows = 8;   // rows at a time

// One block per slot of kBiasRows rows and strip of 256 columns of grad_y.  A
// thread owns 8 columns and every 8th row; the column sums of the block are
// added in a fixed order.  gz is rounded to bf16, the type that both products
// multiply, once and from float32.  Bound by HBM: 32768 rows of 2 x 1024 (335 MB) 70 us, 4.8
// TB/s; 4084 rows of 1000 (24.5 MB) 11 us, of which any launch takes 4.
__global__ __launch_bounds__(kActCols * kActRows) void expert_act_grad_kernel(
    ExpertDims x, const int32_t* __restrict__ off, const uint16_t* __restrict__ gy,
    const uint16_t* __restrict__ pre, uint16_t* __restrict__ gz, float* __restrict__ partial,
    int band, int64_t base, int64_t total, int strips) {
  __shared__ float s_sum[kActRows][kActCols * 8];
  const int64_t tile = base + blockIdx.x;
  if (tile >= total) return;
  const int slot = off[0] / kBiasRows + (int)(tile / strips);
  const Segment s = segment_of_slot(off, x.E, slot, kBiasRows);
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
  const bool act = x.act != MOE_ACT_NONE;
  if (col < x.N) {
    constexpr int kAhead = 4;  // rows whose loads are issued together
    for (int r = r0; r < s.rows; r += kAhead * kActRows) {
      u32x4 vg[kAhead], vz[kAhead], vu[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t row = s.row + min(r + i * kActRows, s.rows - 1);
        vg[i] = *reinterpret_cast<const u32x4*>(gy + row * x.N + col);
        if (act) vz[i] = *reinterpret_cast<const u32x4*>(pre + row * x.Z + col);
        if (two) vu[i] = *reinterpret_cast<const u32x4*>(pre + row * x.Z + x.N + col);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r + i * kActRows >= s.rows) continue;
        const int64_t row = s.row + r + i * kActRows;
        float g[8], o[8];
        unpack8(vg[i], g);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = g[q];
        if (act) {
          float z[8], value[8], slope[8];
          unpack8(vz[i], z);
          act_slopes(x.act, z, value, slope);
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] *= slope[q];
          if (two) {
            float up[8], u[8];
            unpack8(vu[i], up);
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
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !two) break;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) s_sum[r0][c * 8 + q] = sum[h][q];
    __syncthreads();
    const int n = threadIdx.x;  // one column a thread
    float t = 0.0f;
    for (int r = 0; r < kActRows; ++r) t += s_sum[r][n];
    if (col0 + n < x.N)
      partial[((int64_t)slot + (int64_t)band * x.E) * x.Z + h * x.N + col0 + n] = t;
  }
}

// Launches `total` blocks in ranges of at most kMaxTileBlocks.
template <typename F>
hipError_t in_ranges(int64_t total, F f) {
  hipError_t e = hipSuccess;
  for (int64_t b = 0; b < total && e == hipSuccess; b += kMaxTileBlocks)
    e = f(dim3((uint32_t)std::min(total - b, kMaxTileBlocks)), b);
  return e;
}

constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The kernel for few rows is taken up to kFewRows rows an expert on average,
// and up to twice that where the tiles would leave more than half of the CUs
// without one.  Its passes take 16 rows up to half of kFewRows (or where no
// expert can have more), else 32.  Measured, few rows against tiles, 2048 ->
// 1024: gated, 64 experts, top-8: 1 token 13.3 and 29.5 us, 16 tokens 85.9 and
// 112.8, 64 tokens 116.5 and 125.5, 128 tokens 134.4 and 126.5; not gated, 8
// experts, top-2, 64 tokens 12.0 and 29.7; 16 rows a pass against 32: 64
// experts, 32 tokens 98.4 and 102.3 us.
constexpr int kFewRows = 8;

bool few_rows(const ExpertDims& x) {
  const int64_t most = (int64_t)x.E * kFewRows;
  const int tiles = ceil_div(x.N, gated(x.act) ? 128 : 256);
  return x.rows <= most || (x.rows <= 2 * most && (int64_t)x.E * tiles <= kCus / 2);
}

// Large tiles for the weight gradient where every CU gets at least four of them
// (64 experts, 4096 tokens, top-8, 2048 x 2048: 347 us against 365; 1021 tokens,
// 1000 x 776, 480 tiles: 23.4 us against 22.6; one expert of 32768 rows, 64 tiles:
// 745 against 497).
bool large_weight_tiles(const ExpertDims& x) {
  return (int64_t)x.E * ceil_div(x.Z, 256) * ceil_div(x.K, 256) >= 4 * kCus;
}

// Blocks for the row products: the most row tiles there can be are
// rows / BM + E (the counts are only known on the device).
template <typename P>
dim3 row_blocks(const ExpertDims& x, int ntiles) {
  const TileGrid<P::BM, P::BN> most(1, x.rows / P::BM + x.E, ntiles);
  return dim3(std::min(most.numbers(), blocks_at_once<P>()));
}

// Calls f(sizes, offsets, band) for every band: its rows as a product of its own.
template <typename F>
hipError_t by_band(const ExpertDims& x, const int32_t* off, F f) {
  hipError_t e = hipSuccess;
  for (int b = 0; b < x.bands && e == hipSuccess; ++b) {
    ExpertDims xb = x;
    if (x.bands > 1) {
      xb.T = std::min(x.band_tokens, x.T - b * x.band_tokens);
      xb.rows = x.rows / x.T * xb.T;
    }
    e = f(xb, off + (int64_t)b * (x.E + 1), b);
  }
  return e;
}

template <typename T>
struct Type {
  using type = T;
};

template <int BM, int WM, bool GATED>
using RowsTile = TileProduct<BM, 256, WM, 4, false, false, GATED>;
template <int BM, int WM>
using RowsGradTile = TileProduct<BM, 256, WM, 4, false, true, false>;
template <int BM, int WM>
using WgradTile = TileProduct<BM, 256, WM, 4, true, true, false>;

}  // namespace

namespace {

hipError_t expert_rows(const ExpertDims& x, const int32_t* off, const uint16_t* a,
                       const uint16_t* w, const float* bias, const uint16_t* residual, uint16_t* y,
                       uint16_t* pre, hipStream_t s) {
  auto few = [&](auto kernel) {
    const int strips = ceil_div(x.N, 16);
    return in_ranges((int64_t)std::min(x.E, x.rows) * strips, [&](dim3 blocks, int64_t b) {
      return launch(MOE_KERNEL_EXPERT_FEW_ROWS, kernel, blocks, dim3(kFewWaves * kWave), 0, s, x, off,
                    reinterpret_cast<const char*>(a), reinterpret_cast<const char*>(w), bias, residual,
                    y, pre, strips, b);
    });
  };
  if (few_rows(x)) {
    if (x.T <= 16 || (int64_t)x.rows <= (int64_t)x.E * (kFewRows / 2))
      return gated(x.act) ? few(expert_few_rows_kernel<1, true>) : few(expert_few_rows_kernel<1, false>);
    return gated(x.act) ? few(expert_few_rows_kernel<2, true>) : few(expert_few_rows_kernel<2, false>);
  }
  auto go = [&](auto tile) {
    using P = typename decltype(tile)::type;
    const int ntiles = ceil_div(x.N, P::GATED ? P::BN / 2 : P::BN);
    return launch(MOE_KERNEL_EXPERT_ROWS, expert_rows_kernel<P>, row_blocks<P>(x, ntiles),
                  dim3(P::kThreads), 0, s, x, off, reinterpret_cast<const char*>(a),
                  reinterpret_cast<const char*>(w), bias, residual, y, pre, ntiles);
  };
  // Half as many rows a tile where experts have few (64 experts, 32 rows each:
  // 121 us against 131; 128 rows each: 153 against 146; 512: 378 against 348).
  if ((int64_t)x.rows <= (int64_t)x.E * 64)
    return gated(x.act) ? go(Type<RowsTile<128, 1, true>>()) : go(Type<RowsTile<128, 1, false>>());
  return gated(x.act) ? go(Type<RowsTile<256, 2, true>>()) : go(Type<RowsTile<256, 2, false>>());
}

}  // namespace

hipError_t launch_expert_rows(const ExpertDims& x, const int32_t* off, const uint16_t* a,
                              const uint16_t* w, const float* bias, const uint16_t* residual,
                              uint16_t* y, uint16_t* pre, hipStream_t s) {
  return by_band(x, off, [&](const ExpertDims& xb, const int32_t* ob, int) {
    return expert_rows(xb, ob, a, w, bias, residual, y, pre, s);
  });
}

hipError_t launch_expert_rows_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                                   const uint16_t* w, uint16_t* gx, hipStream_t s) {
  using P = RowsGradTile<128, 1>;
  const int ntiles = ceil_div(x.K, P::BN);
  return by_band(x, off, [&](const ExpertDims& xb, const int32_t* ob, int) {
    return launch(MOE_KERNEL_EXPERT_ROWS_GRAD, expert_rows_grad_kernel<P>, row_blocks<P>(xb, ntiles),
                  dim3(P::kThreads), 0, s, xb, ob, reinterpret_cast<const char*>(gz),
                  reinterpret_cast<const char*>(w), gx, ntiles);
  });
}

hipError_t launch_expert_wgrad(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                               const uint16_t* a, void* gw, bool f32, hipStream_t s) {
  auto go = [&](auto tile) {
    using P = typename decltype(tile)::type;
    const TileGrid<P::BM, P::BN> grid(x.E, ceil_div(x.Z, P::BM), ceil_div(x.K, P::BN));
    return launch(MOE_KERNEL_EXPERT_WGRAD,
                  f32 ? expert_wgrad_kernel<P, true> : expert_wgrad_kernel<P, false>,
                  dim3(std::min(grid.numbers(), blocks_at_once<P>())), dim3(P::kThreads), 0, s, x, off,
                  reinterpret_cast<const char*>(gz), reinterpret_cast<const char*>(a), gw, grid);
  };
  if (large_weight_tiles(x)) return go(Type<WgradTile<256, 2>>());
  return go(Type<WgradTile<128, 1>>());
}

// Both gradients in one launch, so that the few blocks that one of them has left
// at its end run beside the other's.  Both in tiles of 256 rows where the weight
// gradient takes those on its own, else both in tiles of 128 (a launch has one
// size of block).  Apart and together, in us: 1021 tokens, 30 experts, top-4,
// 776 -> 1000: 43.6, 36.5; 64 experts, top-8, 2048 -> 1024 gated, 256 tokens: 275,
// 235; 1024: 343, 305; 2048: 426, 428; 4096: 672, 653; 8192 uneven tokens, 128
// experts, 1024 -> 4096: 1490, 1391.  Tiles of 128 in the large launches: 256
// tokens 225, 1024 tokens 333, 16384 tokens of 8 experts, 4096 x 4096, 2362 against
// 1863.  A plan of several bands computes them apart: its weight gradient takes
// all bands at once, the other goes band by band.  The bias sums join them where
// they are a block a CU at most, ahead of the tiles' blocks, which are fewer on a
// CU than theirs would be in a launch of their own.
hipError_t launch_expert_grads(const ExpertDims& x, const int32_t* off, const uint16_t* gz,
                               const uint16_t* w, uint16_t* gx, const uint16_t* a, void* gw,
                               bool f32, const float* partial, float* gb, hipStream_t s) {
  const int threads = large_weight_tiles(x) ? WgradTile<256, 2>::kThreads : WgradTile<128, 1>::kThreads;
  int64_t bias_blocks = gb != nullptr ? (int64_t)x.E * ceil_div(x.Z, threads) : 0;
  if (x.bands > 1 || bias_blocks > kCus) {
    const hipError_t e = gb != nullptr ? launch_expert_bias_sum(x, off, partial, gb, s) : hipSuccess;
    if (e != hipSuccess) return e;
    bias_blocks = 0;
  }
  if (x.bands > 1) {
    const hipError_t e = launch_expert_wgrad(x, off, gz, a, gw, f32, s);
    return e != hipSuccess ? e : launch_expert_rows_grad(x, off, gz, w, gx, s);
  }
  auto go = [&](auto rows_tile, auto weight_tile) {
    using PR = typename decltype(rows_tile)::type;
    using PW = typename decltype(weight_tile)::type;
    const int ntiles = ceil_div(x.K, PR::BN);
    const TileGrid<PW::BM, PW::BN> grid(x.E, ceil_div(x.Z, PW::BM), ceil_div(x.K, PW::BN));
    const int rb = (int)row_blocks<PR>(x, ntiles).x;
    const int wb = std::min(grid.numbers(), blocks_at_once<PW>());
    return launch(MOE_KERNEL_EXPERT_GRADS,
                  f32 ? expert_grads_kernel<PR, PW, true> : expert_grads_kernel<PR, PW, false>,
                  dim3((int)bias_blocks + rb + wb), dim3(PR::kThreads), 0, s, x, off,
                  reinterpret_cast<const char*>(gz), reinterpret_cast<const char*>(w), gx, ntiles,
                  reinterpret_cast<const char*>(a), gw, grid, partial, gb, rb, (int)bias_blocks);
  };
  if (large_weight_tiles(x)) return go(Type<RowsGradTile<256, 2>>(), Type<WgradTile<256, 2>>());
  return go(Type<RowsGradTile<128, 1>>(), Type<WgradTile<128, 1>>());
}

hipError_t launch_expert_act_grad(const ExpertDims& x, const int32_t* off, const uint16_t* gy,
                                  const uint16_t* pre, uint16_t* gz, float* partial,
                                  hipStream_t s) {
  const int strips = ceil_div(x.N, kActCols * 8);
  return by_band(x, off, [&](const ExpertDims& xb, const int32_t* ob, int band) {
    // a band may start and end inside a slot
    const int64_t total = (xb.rows / kBiasRows + x.E + (x.bands > 1)) * (int64_t)strips;
    return in_ranges(total, [&](dim3 grid, int64_t b) {
      return launch(MOE_KERNEL_EXPERT_ACT_GRAD, expert_act_grad_kernel, grid,
                    dim3(kActCols * kActRows), 0, s, xb, ob, gy, pre, gz, partial, band, b, total,
                    strips);
    });
  });
}

hipError_t launch_expert_bias_sum(const ExpertDims& x, const int32_t* off, const float* partial,
                                  float* gb, hipStream_t s) {
  return launch(MOE_KERNEL_EXPERT_BIAS_SUM, expert_bias_sum_kernel,
                dim3((uint32_t)(x.E * ceil_div(x.Z, kBiasThreads))), dim3(kBiasThreads), 0, s, x, off,
                partial, gb);
}

}  // namespace moe

#include "expert4.h"
