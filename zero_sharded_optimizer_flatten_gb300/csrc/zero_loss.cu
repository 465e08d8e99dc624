// Linear softmax cross entropy over a vocabulary, and its gradients, without
// the logits in memory. Argument checks, kernels, launches.
//
//   z = scale * x w^T        x [tokens, hidden], w [vocab, hidden]
//   lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target(t)
//   dz_tv = g_t (exp(z_tv - lse_t) - [v = target(t)])
//   dx = scale * dz w,  dw = scale * dz^T x
//
// Tokens whose target lies outside [0, vocab) are left out: the rows of the
// others are first copied together ("kept rows"), so that all products are
// over them alone and nothing of a left-out row is read.
//
// One kernel (k_loss_product) does the products of both passes:
//   kStats  tiles of z, of which only every row's target and the others'
//           maximum and sum of exponentials leave the SM; joined by k_loss_finish
//           (kStatsLong: for a long depth, summed in several accumulators)
//   kProbs  tiles of z again, to dz in 16 bits, a piece of the vocabulary at a
//           time (kPieceBytes); for dw in binary32 to two 16-bit numbers
//           ("terms"), the second what the first one's rounding lost; of fp16
//           tokens with gradients of their own once more for dx, every row with
//           a scale of its own
//   kGrads  dz w, summed over the pieces in binary32 (kDx), and dz^T x, the
//           piece's rows of dw (kDw), whose tiles fill each other's last round
// The second forming of z is a quarter of the operations: the price of keeping
// no logits between the passes.
//
// Every wait is bounded. One that gives up raises the device error word and the
// call's own flag, which k_loss_gather clears (or raises, while the error word has
// not been reported); k_loss_finish and k_loss_join read it and write NaN.
#include <cuda.h>
#include <cuda_runtime.h>
#include <inttypes.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "zero_capi_util.h"
#include "zero_drain.h"
#include "zero_internal.h"
#include "zero_rows.cuh"
#include "zero_tensor_core.cuh"
#include "zero_windows.cuh"

namespace zero {
namespace {

constexpr int kTileM = 256, kTileN = 256;  // of a pair of CTAs; each holds half of both operands' rows
constexpr int kTileK = 64;                 // 128 bytes of 16-bit data: one swizzled row
constexpr int kHalfRows = 128;
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalfRows * kTileK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = 8;  // two for each quarter of the rows, 128 columns each
constexpr int kThreads = 64 + 32 * kEpilogueWarps;  // copies, products, epilogue
constexpr int kParts = kEpilogueWarps / 4;          // of a row's 256 columns
constexpr int kPartColumns = kTileN / kParts;
constexpr int kAccumulators = 2;
// Blocks of the depth that one accumulator of kStatsLong, and of dw in
// kGradsLong, sums up; they are added up in the epilogue, because the tensor
// cores' additions are rounded less well than binary32 ones. Losses of 4096
// channels are off by 8e-7 of their size in one sum, by 4e-7 in two (of 32
// blocks), by 2e-7 in four, which costs 3% of the time. A binary32 dw of 4096
// tokens, 131072 x 1024, is off by 2.4e-6 in sums of 32 blocks, 8e-7 of 8 and 6e-7
// of 4, which costs 7%.
constexpr int kSegment = 32, kSegmentDw = 8;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes;
constexpr int64_t kPieceBytes = INT64_C(512) << 20;  // of dz in memory at a time
constexpr int kGroupM = 8;  // row tiles that run through the column tiles together (their operands stay in L2)
constexpr int kPairsMost = kSMs / 2;
static_assert(kTileM == kTileN, "rows of w are counted in tiles of either kind");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Product { kStats, kStatsLong, kProbs, kGrads, kGradsLong, kDx, kDw };
constexpr bool is_stats(int kind) { return kind == kStats || kind == kStatsLong; }
constexpr bool is_grads(int kind) { return kind == kGrads || kind == kGradsLong; }
constexpr bool is_z(int kind) { return is_stats(kind) || kind == kProbs; }

// What the host does not know: the kept rows, and what scales them.
struct Scales {
  float mul;    // of dz before it is rounded, a power of two: largest |dz| below 2^14
  float alpha;  // of the products, scale / mul
  float g;      // d_loss as one number (sum, mean)
  int32_t own;  // rows of fp16 have a scale each for dx (see own_scales)
};

// The kept rows, however the caller's list was treated since.
__device__ __forceinline__ int kept_rows(const int32_t* count, int64_t tokens) {
  return min(max(*count, 0), static_cast<int>(tokens));
}

// Where a product goes: rows of `p`, the product's first to row `first`.
struct Out {
  void* p;
  int64_t stride, first;
  int32_t type, align;
};

struct ProductArgs {
  CUtensorMap a, b;    // kGrads: of dx
  CUtensorMap a2, b2;  // kGrads: of dw; kStats, kProbs: b2 for narrow tiles
  const int32_t* count;  // kept rows n
  int64_t rows_cap;      // n rounded up to whole tiles at most
  int32_t hidden;
  int32_t first;         // the piece's first column of z
  int32_t columns;       // of the piece
  int32_t piece;         // columns of a whole piece
  int32_t bf16;
  int32_t *err, *gave_up;
  // kStats, kProbs
  int32_t narrow;        // columns of a narrow tile
  int32_t rows_a;        // rows of x in a box (fewer than 128: of one CTA, there are no more)
  float scale2;          // scale * log2(e)
  const int32_t* target;
  float2* part;          // [column tiles * 2][n rounded up]: maximum and sum without the target's, base 2
  float* target_z;       // base 2
  const float* lse2;
  const float* row_mul;
  const float* row_own;  // or null: dz once more, times this, behind the terms (if scales say so)
  const float* rest;     // 1 - p of the targets, or null: from lse2
  void* dz;              // [terms (+ 1)][rows_cap][dz_stride]
  int64_t dz_stride;
  int32_t terms;
  // kDx, kDw
  const Scales* scales;
  const float* row_alpha;  // kDx: the rows', or null: scales'
  const int32_t* rows;   // kept row -> token
  int64_t tokens;
  Out dx, dw;  // p null: not wanted
  float* sums;           // kDx: [splits][n rounded up][sums_stride]
  int64_t sums_stride;
  int32_t add, pieces, pairs;
  int32_t direct;  // kDx: dx may be written by the product (when its sum has one part)
};

__host__ __device__ __forceinline__ int64_t up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
__host__ __device__ __forceinline__ int64_t over(int64_t n, int64_t unit) { return (n + unit - 1) / unit; }

// How many parts kDx's sum over the vocabulary is cut into, so that few row
// tiles still fill the SMs (their sums are joined by k_loss_join).
__host__ __device__ __forceinline__ int split_of(int tiles, int depth, int pairs) {
  if (tiles < 1 || tiles * 2 > pairs) return 1;
  const int most = (depth + 4 * kTileK - 1) / (4 * kTileK), s = pairs / tiles;
  return s < most ? s : most;
}

// Columns of z that a tile takes. With few tiles the pairs' last round is mostly
// empty: narrower tiles fill it (the eight rows of 4096 against 32000 columns:
// 143 tiles of 224 on 76 pairs in place of 125 of 256). Above two rounds the
// narrower tile's extra reads of x cost as much as it gains. The host chooses
// the narrow width for as many rows as there can be, the device between it and
// the whole one for those that are kept.
// (32-bit numbers: 64-bit divisions in every thread of k_loss_finish took 2 us.)
__host__ __device__ __forceinline__ int tile_cost(int m_tiles, int columns, int tile, int pairs) {
  return (m_tiles * ((columns + tile - 1) / tile) + pairs - 1) / pairs * tile;
}
inline int narrow_columns(int64_t m_tiles, int64_t columns, int pairs) {
  if (m_tiles * over(columns, kTileN) > 2 * pairs) return kTileN;  // so their product below is small
  const int m = static_cast<int>(m_tiles), n = static_cast<int>(columns);
  int best = kTileN;
  for (int t = kTileN - 32; t > kTileN / 2; t -= 32)
    if (tile_cost(m, n, t, pairs) < tile_cost(m, n, best, pairs)) best = t;
  return best;
}
__device__ __forceinline__ int tile_columns(int m_tiles, int columns, int narrow, int pairs) {
  if (narrow == kTileN) return kTileN;
  return tile_cost(m_tiles, columns, narrow, pairs) < tile_cost(m_tiles, columns, kTileN, pairs) ? narrow : kTileN;
}

// The tiles of a product and their order. (All in 32 bits: there are at most
// 2^16 x 2^14 tiles, and a 64-bit division costs as much as a block's products.)
template <int KIND>
struct Tiles {
  int m_tiles, n_tiles, splits, depth_blocks, columns, total;
  __device__ __forceinline__ Tiles(const ProductArgs& a, int n) {
    const int rows = KIND == kDw ? a.columns : n;
    const int cols = KIND == kDx || KIND == kDw ? a.hidden : a.columns;
    const int depth = KIND == kDx ? a.columns : KIND == kDw ? n : a.hidden;
    m_tiles = (rows + kTileM - 1) / kTileM;
    columns = is_z(KIND) ? tile_columns(m_tiles, cols, a.narrow, a.pairs) : kTileN;
    n_tiles = (cols + columns - 1) / columns;
    depth_blocks = (depth + kTileK - 1) / kTileK * (KIND == kDw ? a.terms : 1);
    splits = KIND == kDx ? split_of(m_tiles * n_tiles, a.piece, a.pairs) : 1;
    total = m_tiles * n_tiles * splits;
  }
  __device__ __forceinline__ void at(int t, int& m, int& n, int& s) const {
    s = 0;
    if (KIND == kDx && splits > 1) {
      const int plane = m_tiles * n_tiles;
      s = t / plane;
      t -= s * plane;
    }
    const int group = kGroupM * n_tiles, g = t / group;
    t -= g * group;
    const int m0 = g * kGroupM, size = min(kGroupM, m_tiles - m0);
    n = t / size;
    m = m0 + t - n * size;
  }
  __device__ __forceinline__ void depth(int s, int& k0, int& k1) const {
    k0 = KIND == kDx ? depth_blocks * s / splits : 0;
    k1 = KIND == kDx ? depth_blocks * (s + 1) / splits : depth_blocks;
  }
};

struct Tile {
  int m, n, s, k0, k1;
  bool dw;
};

// The tiles of one pair, one after the other: every `pairs`-th.
template <int KIND>
struct Schedule {
  Tiles<KIND> tiles;
  int at, pairs;
  __device__ __forceinline__ Schedule(const ProductArgs& a, int n, int pair, int pairs_)
      : tiles(a, n), at(pair), pairs(pairs_) {}
  __device__ __forceinline__ int columns() const { return tiles.columns; }
  __device__ __forceinline__ bool next(Tile& t) {
    if (at >= tiles.total) return false;
    tiles.at(at, t.m, t.n, t.s);
    tiles.depth(t.s, t.k0, t.k1);
    t.dw = false;
    at += pairs;
    return true;
  }
};

// The deeper of dx's and dw's tiles first. The pairs that have none in their last
// round do as many of the others instead as end first with the rest; then all go
// on with the others. (Two launches: 4% of dx's time and 3% of dw's are idle at
// 8192 x 4096 x 32000, and each has a start and an end.)
struct GradsSchedule {
  Tiles<kDx> dx;
  Tiles<kDw> dw;
  int at, pairs, pair, deep_total, flat_total, idle, ahead, from, stage = 0;
  bool dw_first;
  __device__ __forceinline__ GradsSchedule(const ProductArgs& a, int n, int pair_, int pairs_)
      : dx(a, n), dw(a, n), at(pair_), pairs(pairs_), pair(pair_) {
    if (!a.dx.p) dx.total = 0;
    if (!a.dw.p) dw.total = 0;
    // a tile costs about eight blocks beside its own
    const int of_dx = dx.depth_blocks / dx.splits + 8, of_dw = dw.depth_blocks + 8;
    dw_first = of_dw > of_dx;
    const int deep = max(of_dx, of_dw), flat = min(of_dx, of_dw);
    deep_total = dw_first ? dw.total : dx.total, flat_total = dw_first ? dx.total : dw.total;
    const int busy = deep_total % pairs;
    idle = busy ? pairs - busy : 0;
    int least = INT32_MAX, best = 0;
    for (int each = deep / flat, k = 0; k < 3 && idle; ++k, ++each) {
      const int64_t end = max(deep, each * flat) + static_cast<int64_t>((max(0, flat_total - each * idle) + pairs - 1) / pairs) * flat;
      if (end < least) least = static_cast<int>(end), best = each;
    }
    ahead = static_cast<int>(min(static_cast<int64_t>(flat_total), static_cast<int64_t>(best) * idle));
    from = pair - busy;  // among the idle ones
  }
  __device__ __forceinline__ int columns() const { return kTileN; }
  __device__ __forceinline__ void take(bool of_dw, Tile& t) const {
    t.dw = of_dw;
    if (of_dw) {
      dw.at(at, t.m, t.n, t.s);
      dw.depth(t.s, t.k0, t.k1);
    } else {
      dx.at(at, t.m, t.n, t.s);
      dx.depth(t.s, t.k0, t.k1);
    }
  }
  __device__ __forceinline__ bool next(Tile& t) {
    if (stage == 0) {
      if (at < deep_total) {
        take(dw_first, t);
        at += pairs;
        return true;
      }
      stage = 1;
      at = idle && from >= 0 ? from : ahead;
    }
    if (stage == 1 && at >= ahead) stage = 2, at = ahead + pair;
    if (at >= flat_total) return false;
    take(!dw_first, t);
    at += stage == 1 ? idle : pairs;
    return true;
  }
};
template <>
struct Schedule<kGrads> : GradsSchedule {
  using GradsSchedule::GradsSchedule;
};
template <>
struct Schedule<kGradsLong> : GradsSchedule {
  using GradsSchedule::GradsSchedule;
};

// A phase-counting position in a ring of `size` slots.
template <int SIZE>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SIZE) slot = 0, phase ^= 1;
  }
};

// 32 consecutive values of a row, `left` of them inside it.
__device__ __forceinline__ void store_words(uint32_t* p, const uint32_t* w, int words, int align) {
  if (align >= 32) {
#pragma unroll
    for (int i = 0; i < words; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i), "r"(w[i]), "r"(w[i + 1]),
                   "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < words; i += 4)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}
template <class T>
__device__ __forceinline__ void store32(T* p, const float (&v)[32], int left, int align) {
  if (left >= 32 && align >= 16) {
    if constexpr (sizeof(T) == 4) {
      store_words(reinterpret_cast<uint32_t*>(p), reinterpret_cast<const uint32_t*>(v), 32, align);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = Elem<T>::pack(v[2 * i], v[2 * i + 1]);
      store_words(reinterpret_cast<uint32_t*>(p), w, 16, align);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < left) p[i] = Elem<T>::narrow(v[i]);
  }
}

// A warp's part of a tile's epilogue, a row a thread: up to 128 columns, 32 at a
// time, from tensor memory.
template <int KIND, bool WIDE = false>  // WIDE: to binary32
struct Epilogue {
  const ProductArgs& a;
  int n;            // kept rows
  int64_t row;      // of the product
  int col, split;
  int64_t part;     // kStats: which of the row's parts this is

  // maximum and sum of exponentials so far
  float top = -INFINITY, sum = 0.f;
  int target = -1;
  float lse2 = 0.f, mul = 0.f, own = 0.f, rest = 0.f;
  float alpha = 0.f;
  int64_t token = -1;
  bool direct = true, twice;
  int64_t sums_rows = 0;

  __device__ __forceinline__ Epilogue(const ProductArgs& a_, int n_, const Tiles<KIND>& t, int m, int nt, int split_,
                                      int row_in_tile, int half, bool twice_)
      : a(a_), n(n_), split(split_), twice(twice_) {
    row = static_cast<int64_t>(m) * kTileM + row_in_tile;
    col = nt * t.columns;
    part = nt * INT64_C(1) * kParts + half;
    const bool live = KIND == kDw ? row < a.columns : row < n;
    if constexpr (is_z(KIND)) {
      if (live) target = a.target[row] - a.first;
    }
    if constexpr (KIND == kProbs) {
      if (live) lse2 = a.lse2[row], mul = a.row_mul[row];
      if (live && a.rest) rest = a.rest[row];
      if (live && twice) own = a.row_own[row];
    }
    if constexpr (KIND == kDx) {
      direct = a.direct && a.pieces == 1 && t.splits == 1;
      sums_rows = up(n, kTileM);
      if (live) token = a.rows[row];
      if (token >= a.tokens) token = -1;  // negative ones are not written either
      alpha = !a.row_alpha ? a.scales->alpha : live ? a.row_alpha[row] : 0.f;
    }
    if constexpr (KIND == kDw) {
      if (live) token = a.dw.first + row;
      alpha = a.scales->alpha;
    }
    (void)live;
  }

  template <class T>
  __device__ __forceinline__ void store_dz(T* to, float (&p)[32]) {
    store32(to, p, 32, 32);
    if (a.terms == 2) {
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i] -= Elem<T>::widen(Elem<T>::narrow(p[i]));
      store32(to + a.rows_cap * a.dz_stride, p, 32, 32);
    }
  }

  // 32 values of z, unscaled, from column c on
  __device__ __forceinline__ void stats(float (&t)[32], int c) {
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] *= a.scale2;
    if (c + 32 > a.columns) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i >= a.columns) t[i] = -INFINITY;
    }
    // the target stands apart: a sum with its 1 in it would lose what a confident
    // token's loss consists of
    const int rel = target - c;
    if (__any_sync(kFull, rel >= 0 && rel < 32)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (rel == i) a.target_z[row] = t[i], t[i] = -INFINITY;
    }
    float most = t[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) most = fmaxf(most, t[i]);
    most = fmaxf(top, most);
    // no finite value yet: nothing to scale (and nothing but zeros to add)
    const float base = most == -INFINITY ? 0.f : most;
    float s = sum * tc::exp2_of(top - base);
#pragma unroll
    for (int i = 0; i < 32; ++i) s += tc::exp2_of(t[i] - base);
    sum = s, top = most;
  }

  __device__ __forceinline__ void take(const uint32_t (&w)[32], int c0, bool zero) {
    const int c = col + c0;
    if constexpr (is_stats(KIND)) {
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = __uint_as_float(w[i]);
      stats(t, c);
    } else if constexpr (KIND == kProbs) {
      if (c >= a.dz_stride) return;  // the last of narrower tiles may pass the piece
      float p[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i] = tc::exp2_of(fmaf(__uint_as_float(w[i]), a.scale2, -lse2));
      const int rel = target - c;
      if (__any_sync(kFull, rel >= 0 && rel < 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (rel == i) p[i] = a.rest ? -rest : p[i] - 1.f;
      }
      if (row >= n) {
#pragma unroll
        for (int i = 0; i < 32; ++i) p[i] = 0.f;
      }
      if (twice) {  // fp16
        float q[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i] = p[i] * own;
        store32(static_cast<__half*>(a.dz) + (a.terms * a.rows_cap + row) * a.dz_stride + c, q, 32, 32);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i] *= mul;
      if (a.bf16)
        store_dz(static_cast<__nv_bfloat16*>(a.dz) + row * a.dz_stride + c, p);
      else
        store_dz(static_cast<__half*>(a.dz) + row * a.dz_stride + c, p);
    } else {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = zero ? 0.f : __uint_as_float(w[i]);
      write(v, c);
    }
  }

  // 32 values of dx or dw, unscaled, from column c on
  __device__ __forceinline__ void write(float (&v)[32], int c) {
    const int left = a.hidden - c;
    if (left <= 0) return;
    if (KIND == kDx && !direct) {
      if (row >= n) return;
      float* p = a.sums + (split * sums_rows + row) * a.sums_stride + c;
      if (a.add) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < left) v[i] += p[i];
      }
      store32(p, v, left, 16);
      return;
    }
    if (token < 0) return;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= alpha;
    const Out& out = KIND == kDx ? a.dx : a.dw;
    const int64_t at = token * out.stride + c;
    if (WIDE || out.type == ZERO_FP32)
      store32(static_cast<float*>(out.p) + at, v, left, out.align);
    else if (out.type == ZERO_BF16)
      store32(static_cast<__nv_bfloat16*>(out.p) + at, v, left, out.align);
    else
      store32(static_cast<__half*>(out.p) + at, v, left, out.align);
  }

  // columns [c0, c1) of the tile, of this warp's rows at d
  __device__ __forceinline__ void run(uint32_t d, int c0, int c1, bool zero) {
    for (int c = c0; c < c1; c += 32) {
      uint32_t w[32];
      tc::tmem_load(d + c, w);
      tc::tmem_wait_load();
      take(w, c, zero);
    }
    done();
  }
  __device__ __forceinline__ void done() {
    if constexpr (is_stats(KIND)) a.part[part * up(n, kTileM) + row] = make_float2(top, sum);
  }

  // the same of a sum in several accumulators: next() gives the place of each
  // (false: given up), free() hands it back
  template <class Next, class Free>
  __device__ __forceinline__ bool run_segments(int segments, int c0, int c1, bool zero, Next next, Free free) {
    constexpr int kChunks = kPartColumns / 32;
    float z[kChunks][32];
    for (int q = 0; q < segments; ++q) {
      uint32_t d;
      if (!next(d)) return false;
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
        if (c0 + 32 * k < c1) {
#pragma unroll
          for (int h = 0; h < 32; h += 16) {  // by 16: what is loaded and the sums fill the registers
            uint32_t w[16];
            tc::tmem_load16(d + c0 + 32 * k + h, w);
            tc::tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float v = zero ? 0.f : __uint_as_float(w[i]);
              z[k][h + i] = q ? z[k][h + i] + v : v;
            }
          }
        }
      free();
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      if (c0 + 32 * k < c1) {
        if constexpr (is_stats(KIND))
          stats(z[k], col + c0 + 32 * k);
        else
          write(z[k], col + c0 + 32 * k);
      }
    done();
    return true;
  }
};

// A persistent pair of CTAs a tile of 256 x 256: one thread of each CTA copies
// its half of the operands' blocks into a ring of kStages, one thread of the
// leading CTA issues the products of both, and eight warps of each CTA work on
// its half of a finished tile in tensor memory while the next one is formed in
// the other accumulator. Where a wait gives up, the products issued so far and the
// copies in flight are waited for before the pair leaves its memory.
template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_loss_product(const __grid_constant__ ProductArgs a) {
  extern __shared__ char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kAccumulators + 1];
  __shared__ uint32_t tmem_slot, stopped;     // stopped: a wait of the pair gave up
  __shared__ __align__(8) uint64_t issued_by[2];  // in the leading CTA: copies of each
  const uint32_t base = (tc::smem_of(raw) + 1023) & ~1023u;
  const uint32_t bar0 = tc::smem_of(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto acc_full = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
  auto acc_empty = [&](int s) { return bar0 + 8u * (2 * kStages + kAccumulators + s); };
  const uint32_t drained = bar0 + 8u * (2 * kStages + 2 * kAccumulators);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();

  let_next_start();
  if (threadIdx.x == 0) {
    tc::prefetch_map(&a.a);
    tc::prefetch_map(&a.b);
    tc::prefetch_map(&a.b2);
    if (is_grads(KIND)) tc::prefetch_map(&a.a2);
    for (int s = 0; s < kStages; ++s) tc::bar_init(full(s), 1), tc::bar_init(empty(s), 1);
    for (int s = 0; s < kAccumulators; ++s) tc::bar_init(acc_full(s), 1), tc::bar_init(acc_empty(s), 2 * kEpilogueWarps);
    tc::bar_init(drained, 1);
    tc::bar_init_fence();
    stopped = 0;
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_of(&tmem_slot), kAccumulators * kTileN);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_previous();

  const bool own = !is_stats(KIND) && a.row_own && a.scales->own;
  const int n = kept_rows(a.count, a.tokens);
  Schedule<KIND> todo(a, n, blockIdx.x >> 1, gridDim.x >> 1);
  Tile t;
  constexpr int kLong = KIND == kGradsLong ? kSegmentDw : kSegment;
  bool ok = true;
  auto give_up = [&] {
    atomicExch(a.err, 1);
    atomicExch(a.gave_up, 1);
    for (uint32_t r = 0; r < 2; ++r) tc::store_cluster(tc::in_cta(tc::smem_of(&stopped), r), 1u);
  };

  if (warp == 0 && lane == 0) {
    // dx's rows of dz
    [[maybe_unused]] const int own_rows =
        is_grads(KIND) && own ? a.terms * static_cast<int>(a.rows_cap) : 0;
    Ring<kStages> ring;
    uint64_t issued = 0;
    while (ok && todo.next(t)) {
      const bool whole = todo.columns() == kTileN;
      // of dw: the depth once for each term of dz, with x again
      [[maybe_unused]] const int depth_end = is_grads(KIND) ? t.k1 / a.terms * kTileK : 0;
      [[maybe_unused]] int depth = 0, term = 0;  // term: its first row of dz
      const int half = todo.columns() / 2;  // of the columns: this CTA's operand rows
      const int row = t.m * kTileM + static_cast<int>(rank) * kHalfRows;
      const int col = t.n * todo.columns() + static_cast<int>(rank) * half;
      const int rows_a = is_grads(KIND) ? kHalfRows : a.rows_a;
      const bool copies_a = rows_a == kHalfRows || rank == 0;
      const uint32_t bytes = static_cast<uint32_t>((rows_a == kHalfRows ? 2 * kHalfRows : rows_a) + todo.columns()) * (kTileK * 2);
      for (int k = t.k0; k < t.k1; ++k) {
        ok = tc::bar_wait(empty(ring.slot), ring.phase ^ 1);
        if (!ok) break;
        const uint32_t to_a = base + ring.slot * kStageBytes, to_b = to_a + kOperandBytes;
        const uint32_t bar = tc::in_cta(full(ring.slot), 0);
        if (rank == 0) tc::bar_expect(full(ring.slot), bytes);
        if (is_grads(KIND) && t.dw) {
          tc::load_box(to_a, &a.a2, row, term + depth, bar);
          tc::load_box(to_a + kOperandBytes / 2, &a.a2, row + 64, term + depth, bar);
          tc::load_box(to_b, &a.b2, col, depth, bar);
          tc::load_box(to_b + kOperandBytes / 2, &a.b2, col + 64, depth, bar);
          depth += kTileK;
          if (depth == depth_end) depth = 0, term += static_cast<int>(a.rows_cap);
        } else if (is_grads(KIND)) {
          tc::load_box(to_a, &a.a, k * kTileK, own_rows + row, bar);
          tc::load_box(to_b, &a.b, col, a.first + k * kTileK, bar);
          tc::load_box(to_b + kOperandBytes / 2, &a.b, col + 64, a.first + k * kTileK, bar);
        } else {
          if (copies_a) tc::load_box(to_a, &a.a, k * kTileK, row, bar);
          // (a map chosen by pointer would be copied to local memory)
          if (whole)
            tc::load_box(to_b, &a.b, k * kTileK, a.first + col, bar);
          else
            tc::load_box(to_b, &a.b2, k * kTileK, a.first + col, bar);
        }
        ++issued;
        ring.next();
      }
    }
    tc::store_cluster(tc::in_cta(tc::smem_of(&issued_by[rank]), 0), issued);
    if (!ok) give_up();
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t kLead = kOperandBytes / 2;
    constexpr bool kBByN = is_grads(KIND);
    const uint32_t plain = tc::instruction(a.bf16 != 0, false, kBByN, kTileM, todo.columns());
    const uint32_t turned = tc::instruction(a.bf16 != 0, true, kBByN, kTileM, todo.columns());
    // 16 deep: 32 bytes along a row, or 16 rows of 128 bytes
    constexpr uint64_t kAlong = 32 >> 4, kAcross = 2048 >> 4;
    Ring<kStages> ring;
    Ring<kAccumulators> acc;
    while (ok && todo.next(t)) {
      ok = tc::bar_wait(acc_empty(acc.slot), acc.phase ^ 1);
      if (!ok) break;
      tc::fence_after();
      const bool a_by_m = is_grads(KIND) && t.dw;
      const uint32_t instr = a_by_m ? turned : plain;
      const uint64_t step_a = a_by_m ? kAcross : kAlong, step_b = kBByN ? kAcross : kAlong;
      uint32_t d = tmem + acc.slot * kTileN;
      int start = t.k0;  // of the sum
      for (int k = t.k0; k < t.k1; ++k) {
        if ((KIND == kStatsLong || (KIND == kGradsLong && t.dw)) && k == start + kLong) {
          tc::commit(acc_full(acc.slot));
          acc.next();
          ok = tc::bar_wait(acc_empty(acc.slot), acc.phase ^ 1);
          if (!ok) break;
          tc::fence_after();
          d = tmem + acc.slot * kTileN;
          start = k;
        }
        ok = tc::bar_wait(full(ring.slot), ring.phase);
        if (!ok) break;
        tc::fence_after();
        const uint32_t at_a = base + ring.slot * kStageBytes, at_b = at_a + kOperandBytes;
        const uint64_t da = tc::operand(at_a, a_by_m ? kLead : 16, 1024);
        const uint64_t db = tc::operand(at_b, kBByN ? kLead : 16, 1024);
#pragma unroll
        for (int i = 0; i < kTileK / 16; ++i)
          tc::mma(d, da + i * step_a, db + i * step_b, instr, k > start || i > 0);
        tc::commit(empty(ring.slot));
        ring.next();
      }
      if (!ok) break;
      tc::commit(acc_full(acc.slot));
      acc.next();
    }
    // the last products: an epilogue that gives up does not wait for them
    tc::commit_here(drained);
    ok = tc::bar_wait(drained, 0) && ok;
    if (!ok) give_up();
  } else if (warp >= 2) {
    Ring<kAccumulators> acc;
    const int quarter = warp & 3;  // the rows of tensor memory that this warp may read
    const int half = (warp - 2) / 4, c0 = half * kPartColumns, c1 = min(todo.columns(), c0 + kPartColumns);
    const int row = static_cast<int>(rank) * kHalfRows + quarter * 32 + lane;
    auto wait = [&] {
      ok = __all_sync(kFull, tc::bar_wait(acc_full(acc.slot), acc.phase));
      tc::fence_after();
      return ok;
    };
    auto place = [&] { return tmem + acc.slot * kTileN + (static_cast<uint32_t>(quarter * 32) << 16); };
    auto free = [&] {
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive_cluster(tc::in_cta(acc_empty(acc.slot), 0));
      acc.next();
    };
    auto work = [&](auto& e) {
      if (!wait()) return;
      e.run(place(), c0, c1, t.k0 == t.k1);
      free();
    };
    [[maybe_unused]] auto next = [&](uint32_t& d) {
      if (!wait()) return false;
      d = place();
      return true;
    };
    [[maybe_unused]] auto segments = [&] { return max(1, (t.k1 - t.k0 + kLong - 1) / kLong); };
    while (ok && todo.next(t)) {
      if constexpr (KIND == kStatsLong) {
        Epilogue<KIND> e(a, n, todo.tiles, t.m, t.n, t.s, row, half, own);
        e.run_segments(segments(), c0, c1, false, next, free);
      } else if constexpr (!is_grads(KIND)) {
        Epilogue<KIND> e(a, n, todo.tiles, t.m, t.n, t.s, row, half, own);
        work(e);
      } else if (t.dw) {
        Epilogue<kDw, KIND == kGradsLong> e(a, n, todo.dw, t.m, t.n, t.s, row, half, own);
        if constexpr (KIND == kGradsLong)
          e.run_segments(segments(), c0, c1, t.k0 == t.k1, next, free);
        else
          work(e);
      } else {
        Epilogue<kDx> e(a, n, todo.dx, t.m, t.n, t.s, row, half, own);
        work(e);
      }
    }
    if (!ok && lane == 0) give_up();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // no CTA leaves while the other may still write to it
  if (stopped) {       // the same in both
    if (rank == 0 && threadIdx.x == 0) {
      const int half = todo.columns() / 2, rows_b = is_grads(KIND) || a.rows_a == kHalfRows ? kHalfRows : 0;
      const uint32_t others = static_cast<uint32_t>(rows_b + half) * (kTileK * 2);  // bytes of the other CTA's copies
      const Drain d(static_cast<int64_t>(issued_by[0]), static_cast<int64_t>(issued_by[1]), kStages);
      for (int64_t j = d.first; j < d.last; ++j) {
        const uint32_t bar = full(static_cast<int>(j % kStages));
        if (d.announce(j))
          tc::bar_expect(bar, others);
        else if (d.forgo(j))
          tc::bar_count(bar, others);
        tc::bar_wait(bar, static_cast<uint32_t>(j / kStages) & 1);
      }
    }
    tc::cluster_sync();
  }
  tc::fence_after();
  if (warp == 1) tc::tmem_free(tmem, kAccumulators * kTileN);
}

// ---------------------------------------------------------------------------
// the kernels around the products

struct RowsArgs {
  const void* targets;
  int32_t id_bytes, vocab;
  int64_t tokens, hidden;
  int32_t* rows;  // [tokens + 1]: the kept tokens in order; the last entry is their number
  int32_t* ticket;
  int32_t *err, *gave_up;
  // gathering
  const void* x;
  int64_t x_stride, xs_stride, rows_cap;
  void* xs;
  int32_t* target;
  int32_t vec, log_lanes, narrow, pairs;
  // gradients
  const float *lse, *rest;
  const float* d;
  int32_t reduction;
  double scale;
  Scales* scales;
  float *lse2, *row_mul, *row_rest;
  float *row_own, *row_alpha;  // or null: see own_scales
  void* dx;
  // losses
  const float2* part;
  const float* target_z;
  float* cta_sums;  // [CTAs of k_loss_finish]
  float *losses, *lse_out, *rest_out, *total;
};

__device__ __forceinline__ int load_target(const RowsArgs& a, int64_t t) {
  const long long v = a.id_bytes == 4 ? static_cast<const int*>(a.targets)[t] : static_cast<const long long*>(a.targets)[t];
  return v >= 0 && v < a.vocab ? static_cast<int>(v) : -1;
}
// Whether token t0 + i * step is kept, the targets loaded together (a choice of
// their type within the loop would make the loads wait for one another).
template <int N>
__device__ __forceinline__ void load_kept(const RowsArgs& a, int64_t t0, int step, bool (&kept)[N]) {
  long long v[N];
  if (t0 >= a.tokens) {
#pragma unroll
    for (int i = 0; i < N; ++i) kept[i] = false;
    return;
  }
  if (a.id_bytes == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<const int*>(a.targets)[min(t0 + i * step, a.tokens - 1)];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<const long long*>(a.targets)[min(t0 + i * step, a.tokens - 1)];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) kept[i] = t0 + i * step < a.tokens && v[i] >= 0 && v[i] < a.vocab;
}

// The kept tokens, in order: one CTA.
constexpr int kScanThreads = 1024, kScanEach = 8;
__global__ void __launch_bounds__(kScanThreads) k_loss_rows(const RowsArgs a) {
  __shared__ int counts[32];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kScanThreads * kScanEach) {
    // a warp's kScanEach rounds of 32 tokens lie one after the other
    const int64_t w0 = t0 + static_cast<int64_t>(warp) * 32 * kScanEach;
    bool kept[kScanEach];
    unsigned votes[kScanEach];
    int mine = 0;
    load_kept(a, w0 + lane, 32, kept);
#pragma unroll
    for (int i = 0; i < kScanEach; ++i) votes[i] = __ballot_sync(kFull, kept[i]), mine += __popc(votes[i]);
    __syncthreads();
    if (lane == 0) counts[warp] = mine;
    __syncthreads();
    int c = counts[lane], inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    int at = before + __shfl_sync(kFull, inc - c, warp);
#pragma unroll
    for (int i = 0; i < kScanEach; ++i) {
      if (kept[i]) a.rows[at + __popc(votes[i] & ((1u << lane) - 1))] = static_cast<int>(w0 + 32 * i + lane);
      at += __popc(votes[i]);
    }
    before += __shfl_sync(kFull, inc, 31);
  }
  for (int64_t t = before + threadIdx.x; t < a.tokens; t += kScanThreads) a.rows[t] = -1;
  if (threadIdx.x == 0) {
    a.rows[a.tokens] = before;
    *a.ticket = 0;
  }
}

// What the gradients are scaled with: every row's g times a power of two that
// brings the largest finite one (`top`) to [2^13, 2^14), so that neither rounding
// to 16 bits nor fp16's range costs small probabilities. A row whose g is infinite
// or NaN stays that, whatever it is scaled with.
__device__ __forceinline__ Scales scales_for(float top, float g, double scale) {
  int e = 14;
  if (top > 0.f && top <= FLT_MAX)
    frexpf(top, &e);
  e = max(e, -100);
  return {ldexpf(1.f, 14 - e), static_cast<float>(ldexp(scale, e - 14)), g, 0};
}
// The one of a sum or a mean; of the tokens' own gradients it takes a pass.
__device__ __forceinline__ Scales scales_of_one(const RowsArgs& a, int n) {
  float g = *a.d;
  if (a.reduction == ZERO_LOSS_MEAN) g = g / static_cast<float>(max(n, 1));
  return scales_for(fabsf(g), g, a.scale);
}
__global__ void __launch_bounds__(kScanThreads) k_loss_scales(const RowsArgs a) {
  __shared__ float most[32], fewest[32];
  let_next_start();
  const int n = kept_rows(a.rows + a.tokens, a.tokens);
  float top = 0.f, low = FLT_MAX;
  for (int i = threadIdx.x; i < n; i += kScanThreads) {
    const int t = a.rows[i];
    const float g = t >= 0 && t < a.tokens ? fabsf(a.d[t]) : 0.f;
    if (g > 0.f && g <= FLT_MAX) top = fmaxf(top, g), low = fminf(low, g);
  }
  auto join = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      top = fmaxf(top, __shfl_xor_sync(kFull, top, o)), low = fminf(low, __shfl_xor_sync(kFull, low, o));
  };
  join();
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = top, fewest[threadIdx.x >> 5] = low;
  __syncthreads();
  top = most[threadIdx.x & 31], low = fewest[threadIdx.x & 31];
  join();
  if (threadIdx.x == 0) {
    Scales s = scales_for(top, 0.f, a.scale);
    s.own = a.row_alpha && low * 65536.f < top;
    *a.scales = s;
  }
}

// Rows to another stride: w to one that the bulk copies can take, dw back from
// one that whole words can be stored to. CTAs of another kernel do it beside its
// own work.
struct CopyArgs {
  const void* from;
  void* to;
  int64_t from_stride, to_stride, rows;
  int32_t hidden, log_lanes, words;  // words: 16-bit ones of an element
  int64_t ctas;
};
// By 16-byte pieces of the row that is written, four in flight; `inner` keeps the
// reads of a row that may begin or end its storage within it. (Single columns:
// 163 us for 38759 rows of 4271 bf16 to padded ones and 263 back, in place of
// 117 and 130, 0.8 of what a plain copy of them takes.)
template <class T>
__device__ __forceinline__ void copy_row(const T* from, T* to, int hidden, bool inner, int lane, int lanes) {
  const Frame<T> f(to, hidden, inner, inner);
  const int shift = Window<T>::shift(from + f.head);
  for (int u = lane; u < f.pieces; u += 4 * lanes) {
    Window<T> v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k].load(from + f.column(min(u + k * lanes, f.pieces - 1)));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (u + k * lanes < f.pieces) v[k].shifted(shift).store(to + f.column(u + k * lanes));
  }
  for (int e = lane; e < f.ends; e += lanes) to[f.end_column(e)] = from[f.end_column(e)];
}
__device__ __forceinline__ void copy_rows(const CopyArgs& a, int64_t cta) {
  const int lanes = 1 << a.log_lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t i = (cta * blockDim.x + threadIdx.x) >> a.log_lanes;
  if (i >= a.rows) return;
  const bool inner = i == 0 || i == a.rows - 1;
  if (a.words == 2)
    copy_row(static_cast<const float*>(a.from) + i * a.from_stride, static_cast<float*>(a.to) + i * a.to_stride,
             a.hidden, inner, lane, lanes);
  else
    copy_row(static_cast<const __half*>(a.from) + i * a.from_stride, static_cast<__half*>(a.to) + i * a.to_stride,
             a.hidden, inner, lane, lanes);
}

// The kept rows copied together, in the gradients with zeros up to a whole block
// of the depth of dz^T x; their targets (and what scales them); left-out rows of
// dx. A group of 8 to 256 lanes has a row. The first CTAs copy w, if it takes that.
constexpr int kGatherThreads = 256;
constexpr int kFewTokens = 4 * kGatherThreads;  // whose list every CTA makes for itself: one launch less
enum Gather { kForward, kForwardFew, kBackward };

template <class W, Gather KIND>
__global__ void __launch_bounds__(kGatherThreads) k_loss_gather(const RowsArgs a, const CopyArgs copy) {
  constexpr bool BACKWARD = KIND == kBackward;
  __shared__ int few[KIND == kForwardFew ? kFewTokens : 1], counts[kGatherThreads / 32];
  let_next_start();
  wait_for_previous();
  if (blockIdx.x < copy.ctas) {
    copy_rows(copy, blockIdx.x);
    return;
  }
  const int64_t cta = blockIdx.x - copy.ctas;
  const bool first = cta == 0 && threadIdx.x == 0;
  const int err = first ? *a.err : 0;  // stored at the end: nothing waits for it
  int n;
  if constexpr (KIND == kForwardFew) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool kept[4];
    unsigned votes[4];
    load_kept(a, warp * 128 + lane, 32, kept);
    int mine = 0, at = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) votes[k] = __ballot_sync(kFull, kept[k]), mine += __popc(votes[k]);
    if (lane == 0) counts[warp] = mine;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kGatherThreads / 32; ++w) {
      if (w < warp) at += counts[w];
      n += counts[w];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (kept[k]) few[at + __popc(votes[k] & ((1u << lane) - 1))] = warp * 128 + 32 * k + lane;
      at += __popc(votes[k]);
    }
    __syncthreads();
    if (cta == 0) {
      for (int k = threadIdx.x; k < a.tokens; k += kGatherThreads) a.rows[k] = k < n ? few[k] : -1;
      if (threadIdx.x == 0) a.rows[a.tokens] = n, *a.ticket = 0;
    }
  } else {
    n = kept_rows(a.rows + a.tokens, a.tokens);
  }
  [[maybe_unused]] Scales scales = {};
  if constexpr (BACKWARD) {
    if (a.reduction == ZERO_LOSS_NONE) {
      scales = *a.scales;
    } else {
      scales = scales_of_one(a, n);
      if (cta == 0 && threadIdx.x == 0) *a.scales = scales;
    }
  }
  const int lanes = 1 << a.log_lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t i = (cta * kGatherThreads + threadIdx.x) >> a.log_lanes;
  const int words = static_cast<int>(a.hidden * 2 / sizeof(W));
  W* to = reinterpret_cast<W*>(static_cast<char*>(a.xs) + i * a.xs_stride * 2);
  const int t = i >= n ? -1 : KIND == kForwardFew ? few[i] : a.rows[i];
  if (t >= 0 && t < a.tokens) {
    const W* from = reinterpret_cast<const W*>(static_cast<const char*>(a.x) + t * a.x_stride * 2);
    // one lane's, loaded ahead of the row
    int target = -1;
    [[maybe_unused]] float lse = 0.f, rest = 0.f, g = scales.g;
    if (lane == 0) {
      target = load_target(a, t);
      if constexpr (BACKWARD) {
        lse = a.lse[t];
        if (a.rest) rest = a.rest[t];
        if (a.reduction == ZERO_LOSS_NONE) g = a.d[t];
      }
    }
    if constexpr (sizeof(W) == 2) {  // rows that start anywhere
      copy_row(reinterpret_cast<const __half*>(from), reinterpret_cast<__half*>(to), words, t == 0 || t == a.tokens - 1,
               lane, lanes);
    } else {
      for (int c = lane; c < words; c += 4 * lanes) {
        W v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = from[min(c + k * lanes, words - 1)];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k * lanes < words) to[c + k * lanes] = v[k];
      }
    }
    if (lane == 0) {
      a.target[i] = target;
      if constexpr (BACKWARD) {
        a.lse2[i] = lse * kLog2e;
        a.row_mul[i] = target < 0 ? 0.f : g * scales.mul;
        if (a.rest) a.row_rest[i] = rest;
        if (a.row_alpha) {
          const Scales own = scales.own ? scales_for(fabsf(g), g, a.scale) : scales;
          (a.row_own ? a.row_own : a.row_mul)[i] = target < 0 ? 0.f : g * own.mul;
          a.row_alpha[i] = own.alpha;
        }
      }
    }
  } else if (i < n || (BACKWARD && i < up(n, kTileK))) {
    for (int c = lane; c < words; c += lanes) to[c] = W();
    if (lane == 0 && i < n) {
      a.target[i] = -1;
      if constexpr (BACKWARD) {
        a.lse2[i] = 0.f, a.row_mul[i] = 0.f;
        if (a.rest) a.row_rest[i] = 0.f;
        if (a.row_own) a.row_own[i] = 0.f;
        if (a.row_alpha) a.row_alpha[i] = 0.f;
      }
    }
  }
  if constexpr (BACKWARD) {
    if (a.dx && i < a.tokens && load_target(a, i) < 0) {
      W* out = reinterpret_cast<W*>(static_cast<char*>(a.dx) + i * a.hidden * 2);
      for (int c = lane; c < words; c += lanes) out[c] = W();
    }
  }
  if (first) *a.gave_up = err != 0;
}

// Statistics of parts of a row, base 2: the larger maximum, the sum under it.
__device__ __forceinline__ void join(float& top, float& sum, float other_top, float other_sum) {
  const float most = fmaxf(top, other_top), base = most == -INFINITY ? 0.f : most;
  sum = sum * tc::exp2_of(top - base) + other_sum * tc::exp2_of(other_top - base);
  top = most;
}

// Every kept row's statistics joined over its parts, 32 threads a row, and with
// its target; the CTA that is last adds the losses up, in one order.
constexpr int kFinishRows = 8, kFinishGroups = 32, kFinishThreads = kFinishRows * kFinishGroups, kFinishAhead = 8;
__global__ void __launch_bounds__(kFinishThreads) k_loss_finish(const RowsArgs a) {
  __shared__ float2 part[kFinishGroups][kFinishRows + 1];
  __shared__ float sums[kFinishThreads / 32], mine[kFinishRows];
  __shared__ bool last;
  wait_for_previous();
  const int gave_up = *a.gave_up;
  const int n = kept_rows(a.rows + a.tokens, a.tokens);
  const int parts = kParts * static_cast<int>(over(a.vocab, tile_columns((n + kTileM - 1) / kTileM, a.vocab, a.narrow, a.pairs)));
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kFinishRows, rows = up(n, kTileM);
  // of the row that this thread writes: loaded ahead of the parts
  const int64_t own = i0 + threadIdx.x / kFinishGroups;
  const bool writes = threadIdx.x % kFinishGroups == 0;
  const int token = writes && own < n ? a.rows[own] : -1;
  const float target_z = writes && own < n ? a.target_z[own] : 0.f;
  const bool left_out = writes && own < a.tokens && load_target(a, own) < 0;
  {
    const int r = threadIdx.x % kFinishRows, g = threadIdx.x / kFinishRows;
    float top = -INFINITY, sum = 0.f;
    if (i0 + r < n) {
      const float2* from = a.part + i0 + r;
      for (int v = g; v < parts; v += kFinishAhead * kFinishGroups) {
        float2 p[kFinishAhead];
#pragma unroll
        for (int k = 0; k < kFinishAhead; ++k)
          p[k] = from[min(v + k * kFinishGroups, parts - 1) * rows];
#pragma unroll
        for (int k = 0; k < kFinishAhead; ++k)
          if (v + k * kFinishGroups < parts) join(top, sum, p[k].x, p[k].y);
      }
    }
    part[g][r] = make_float2(top, sum);
  }
  __syncthreads();
  {
    const int r = threadIdx.x / kFinishGroups, g = threadIdx.x % kFinishGroups;  // a warp a row
    float2 p = part[g][r];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      join(p.x, p.y, __shfl_xor_sync(kFull, p.x, o), __shfl_xor_sync(kFull, p.y, o));
    if (g == 0) {
      float loss = 0.f;
      if (own < n && token >= 0) {
        // loss = log(1 + 2^d), d what the others' log2 of the sum is above the
        // target: differences first, so that small losses keep all their bits
        const float log_sum = gave_up ? NAN : log2f(p.y), d = (p.x - target_z) + log_sum, e = exp2f(-fabsf(d)), less = log1pf(e);
        loss = target_z < INFINITY ? fmaf(fmaxf(d, 0.f), kLn2, less) : NAN;
        a.lse_out[token] = fmaf(d > 0.f ? p.x + log_sum : target_z, kLn2, less);
        a.losses[token] = loss;
        // the others' probability, 2^d / (1 + 2^d)
        if (a.rest_out) a.rest_out[token] = target_z < INFINITY ? (d > 0.f ? 1.f : e) / (1.f + e) : NAN;
      }
      mine[r] = loss;
      if (left_out) {
        a.lse_out[own] = 0.f, a.losses[own] = 0.f;
        if (a.rest_out) a.rest_out[own] = 0.f;
      }
    }
  }
  __syncthreads();
  // a CTA's losses, then in the last one the CTAs' sums, each thread's with what
  // its additions lose
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int k = 0; k < kFinishRows; ++k) s += mine[k];
    if (gridDim.x == 1) {
      sums[0] = s;
      last = true;
    } else {
      a.cta_sums[blockIdx.x] = s;
      __threadfence();
      last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  float s = 0.f, lost = 0.f;
  if (gridDim.x == 1) {
    s = threadIdx.x == 0 ? sums[0] : 0.f;
    __syncthreads();
  } else {
    __threadfence();
    const int64_t ctas = gridDim.x;
    for (int64_t t = threadIdx.x; t < ctas; t += 8 * kFinishThreads) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __ldcg(a.cta_sums + min(t + k * kFinishThreads, ctas - 1));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (t + k * kFinishThreads < ctas) {
          const float next = s + v[k];
          lost += fabsf(s) >= fabsf(v[k]) ? (s - next) + v[k] : (v[k] - next) + s;
          s = next;
        }
    }
    if (isfinite(s)) s += lost;
  }
  s = warp_all_sum(s);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int k = 0; k < kFinishThreads / 32; ++k) s += sums[k];
    a.total[0] = s / static_cast<float>(max(n, 1));
    a.total[1] = s;
    a.total[2] = static_cast<float>(n);
  }
}

// A copy alone: of dw between two pieces.
__global__ void __launch_bounds__(kGatherThreads) k_loss_copy(const CopyArgs copy) {
  let_next_start();
  wait_for_previous();
  copy_rows(copy, blockIdx.x);
}

// dx from its binary32 sums, where the product did not write it. The first CTAs
// copy the last rows of dw, if it takes that. After a wait that gave up: NaN for
// all that was to be written, by whichever CTAs there are.
struct JoinArgs {
  const int32_t* rows;
  int64_t tokens;
  const float* sums;
  int64_t sums_stride;
  const Scales* scales;
  const float* row_alpha;
  void *dx, *dw;
  int64_t dw_size;
  const int32_t* gave_up;
  int32_t hidden, piece, pieces, pairs, direct, log_lanes, vec, dw_type;
};
template <class T>
__device__ __forceinline__ void write_nan(const JoinArgs& a) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kGatherThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGatherThreads;
  const int64_t size = a.dx ? kept_rows(a.rows + a.tokens, a.tokens) * static_cast<int64_t>(a.hidden) : 0;
  for (int64_t i = first; i < size; i += step) {
    const int64_t row = i / a.hidden, t = a.rows[row];
    if (t >= 0 && t < a.tokens) static_cast<T*>(a.dx)[t * a.hidden + i - row * a.hidden] = Elem<T>::narrow(NAN);
  }
  for (int64_t i = first; a.dw && i < a.dw_size; i += step) store_any(a.dw, i, a.dw_type, NAN);
}
template <class T>
__global__ void __launch_bounds__(kGatherThreads) k_loss_join(const JoinArgs a, const CopyArgs copy) {
  wait_for_previous();
  const int gave_up = *a.gave_up;
  const int n = kept_rows(a.rows + a.tokens, a.tokens);
  if (gave_up) {
    write_nan<T>(a);
    return;
  }
  if (blockIdx.x < copy.ctas) {
    copy_rows(copy, blockIdx.x);
    return;
  }
  if (!a.dx) return;
  const int splits = split_of((n + kTileM - 1) / kTileM * ((a.hidden + kTileN - 1) / kTileN), a.piece, a.pairs);
  if (splits == 1 && a.pieces == 1 && a.direct) return;
  const int lanes = 1 << a.log_lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t i = ((blockIdx.x - copy.ctas) * kGatherThreads + threadIdx.x) >> a.log_lanes;
  if (i >= n) return;
  const int64_t t = a.rows[i];
  if (t < 0 || t >= a.tokens) return;
  const float alpha = a.row_alpha ? a.row_alpha[i] : a.scales->alpha;
  const int64_t part = up(n, kTileM) * a.sums_stride;
  const float* from = a.sums + i * a.sums_stride;
  T* to = static_cast<T*>(a.dx) + t * a.hidden;
  // eight columns side by side, or `lanes` apart where dx's rows start anywhere
  const int next = a.vec ? 1 : lanes;
  for (int c = a.vec ? 8 * lane : lane; c < a.hidden; c += 8 * lanes) {
    float s[8] = {};
    for (int k = 0; k < splits; k += 4) {
      float v[4][8];
      if (a.vec) {
        Octet<float> o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q].load(from + min(k + q, splits - 1) * part + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q].widen(v[q]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[q][j] = from[min(k + q, splits - 1) * part + min(c + j * next, a.hidden - 1)];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (k + q < splits)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] += v[q][j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] *= alpha;
    if (a.vec) {
      Elem<T>::store8(to + c, s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j * next < a.hidden) to[c + j * next] = Elem<T>::narrow(s[j]);
    }
  }
}

// ---------------------------------------------------------------------------
// host

// Tokens with gradients of their own in fp16: one scale for all would round the
// rows of dx whose gradients lie far below the largest to few bits or none, so
// they get one each once the smallest is below 2^-16 of the largest. (Up to there
// probabilities above 2^-10 keep all their bits and none is off by more than 2^-22,
// which sums over 131072 columns to less than dx's own rounding, 2^-12.) dw's sums
// mix the rows, so it keeps dz with the one scale, and dz is written twice: 168 us
// in place of 150 at 1024 x 1024 x 32000. (bf16 has binary32's exponents.)
bool own_scales(const zero_linear_ce_desc& d, int reduction, const void* dx) {
  return d.dtype == ZERO_FP16 && reduction == ZERO_LOSS_NONE && dx;
}

// Where a call's scratch lies. both: room for dx's dz apart from dw's.
struct Layout {
  int64_t rows_cap, dz_rows, all_rows, columns, pieces, xs_stride, w_stride, sums_stride;
  int64_t xs, w, part, target_z, target, ticket, cta_sums, lse2, row_mul, row_rest, row_own, row_alpha, scales, dz, sums, dw, bytes;
  int terms;   // of dz: 16 (bf16) or 22 (fp16) bits for a dw in binary32
  bool whole;  // rows of dx and dw are whole 16-byte words: the products write them

  Layout(const zero_linear_ce_desc& d, bool repack, bool backward, bool both = false) {
    rows_cap = up(std::max<int64_t>(d.tokens, 1), kTileM);
    whole = d.hidden % 8 == 0;
    columns = up(d.vocab, kTileN);
    terms = d.dw_dtype == ZERO_FP32 ? 2 : 1;
    dz_rows = rows_cap * terms;
    all_rows = dz_rows + (both ? rows_cap : 0);
    if (backward) columns = std::min(columns, std::max<int64_t>(kTileN, kPieceBytes / 2 / all_rows / kTileN * kTileN));
    pieces = over(d.vocab, columns);
    xs_stride = up(d.hidden, 8);
    w_stride = repack ? up(d.hidden, 8) : d.w_stride;
    sums_stride = up(d.hidden, 8);
    int64_t at = 0;
    auto take = [&](int64_t size) {
      const int64_t here = at;
      at = up(at + size, 256);
      return here;
    };
    xs = take(rows_cap * xs_stride * 2);
    w = take(repack ? d.vocab * w_stride * 2 : 0);
    target = take(rows_cap * 4);
    ticket = take(8);  // and the flag of a wait that gave up
    cta_sums = take(backward ? 0 : over(rows_cap, kFinishRows) * 4);
    // kParts a tile and row; tiles narrower than 256 are at most three rounds of the pairs
    part = take(backward ? 0 : std::max(kParts * over(d.vocab, kTileN) * rows_cap, INT64_C(3) * kParts * kPairsMost * kTileM) * 8);
    target_z = take(backward ? 0 : rows_cap * 4);
    lse2 = take(backward ? rows_cap * 4 : 0);
    row_mul = take(backward ? rows_cap * 4 : 0);
    row_rest = take(backward ? rows_cap * 4 : 0);
    row_own = take(backward && d.dtype == ZERO_FP16 ? rows_cap * 4 : 0);
    row_alpha = take(backward && d.dtype == ZERO_FP16 ? rows_cap * 4 : 0);
    scales = take(sizeof(Scales));
    dz = take(backward ? all_rows * columns * 2 : 0);
    // as many rows as there are tokens, or the parts of few: splits x row tiles x
    // column tiles are at most the pairs (see split_of), none where one row tile's
    // columns pass half of them
    const int64_t n_tiles = over(d.hidden, kTileN);
    const int64_t split_rows = 2 * n_tiles > kPairsMost ? 0 : kPairsMost / n_tiles * kTileM;
    sums = take(backward ? (pieces > 1 || !whole ? std::max(split_rows, rows_cap) : split_rows) * sums_stride * 4 : 0);
    dw = take(backward && !whole ? columns * sums_stride * 4 : 0);
    bytes = at;
  }
};

bool wants_repack(const zero_linear_ce_desc& d, const void* w) {
  return d.w_stride % 8 != 0 || !aligned_to(w, 16);
}

// Of any reduction.
int64_t workspace_of(const zero_linear_ce_desc& d, const void* w, bool backward) {
  const bool repack = wants_repack(d, w);
  const int64_t bytes = Layout(d, repack, backward).bytes;
  return backward && d.dtype == ZERO_FP16 ? std::max(bytes, Layout(d, repack, true, true).bytes) : bytes;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Map of a matrix [rows][cols] of 16-bit values; boxes of 64 columns.
bool matrix_map(CUtensorMap* map, const void* p, bool bf16, int64_t cols, int64_t rows, int64_t stride, int box_rows) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kTileK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t steps[2] = {1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs that the device holds at a time.
cudaError_t pairs_of(const void* fn, int* pairs) {
  constexpr int kDevices = 8;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && (*pairs = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kPairsMost);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, fn, &cfg);
  if (e != cudaSuccess) return e;
  *pairs = std::max(1, std::min(*pairs, kPairsMost));
  if (dev < kDevices) known[dev].store(*pairs, std::memory_order_relaxed);
  return cudaSuccess;
}

// Lanes of a row's group, a power of two: 8 to 256, `each` columns a lane.
int lanes_for(int64_t hidden, int each) {
  int log_lanes = 3;
  while (log_lanes < 8 && (static_cast<int64_t>(each) << log_lanes) < hidden) ++log_lanes;
  return log_lanes;
}
int64_t ctas_for(int64_t rows, int log_lanes) { return std::max<int64_t>(1, over(rows, kGatherThreads >> log_lanes)); }

template <class... P>
cudaError_t launch(void (*fn)(P...), int64_t grid, int threads, size_t smem, bool early, cudaStream_t s, P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

template <int KIND>
cudaError_t launch_product(ProductArgs& a, cudaStream_t s) {
  static KernelFacts facts;
  const void* fn = reinterpret_cast<const void*>(&k_loss_product<KIND>);
  cudaError_t e = facts.allow(fn, kSmemBytes, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch(&k_loss_product<KIND>, 2 * static_cast<int64_t>(a.pairs), kThreads, kSmemBytes, true, s,
                static_cast<const ProductArgs>(a));
}

template <Gather KIND>
cudaError_t launch_gather(const RowsArgs& a, const CopyArgs& copy, bool early, cudaStream_t s) {
  static LargeShared large[2];
  auto* fn = a.vec ? &k_loss_gather<uint4, KIND> : &k_loss_gather<uint16_t, KIND>;
  // (before kStats: 2 us of 29 at 1021 x 1001 x 5003; before kProbs it costs 1)
  const cudaError_t e = KIND == kBackward ? cudaSuccess : large[a.vec].ask(reinterpret_cast<const void*>(fn));
  return e != cudaSuccess ? e
                          : launch(fn, copy.ctas + ctas_for(a.rows_cap, a.log_lanes), kGatherThreads, 0, early, s, a, copy);
}

zero_status check_desc(const char* fn, const zero_linear_ce_desc* d) {
  if (!d) return fail(ZERO_ERR_INVALID, "%s: desc is NULL", fn);
  if (d->tokens < 0 || d->tokens > 1 << 24)
    return fail(ZERO_ERR_INVALID, "%s: tokens must lie in [0, 2^24]", fn);
  if (d->hidden < 1 || d->hidden > 1 << 20) return fail(ZERO_ERR_INVALID, "%s: hidden must lie in [1, 2^20]", fn);
  if (d->vocab < 1 || d->vocab > 1 << 22) return fail(ZERO_ERR_INVALID, "%s: vocab must lie in [1, 2^22]", fn);
  if (d->dtype != ZERO_FP16 && d->dtype != ZERO_BF16)
    return fail(ZERO_ERR_INVALID, "%s: dtype must be ZERO_FP16 or ZERO_BF16", fn);
  if (d->dw_dtype != d->dtype && d->dw_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: dw_dtype must be dtype or ZERO_FP32", fn);
  if (d->id_bytes != 4 && d->id_bytes != 8) return fail(ZERO_ERR_INVALID, "%s: id_bytes must be 4 or 8", fn);
  if (!std::isfinite(d->scale) || d->scale == 0.0 || std::fabs(d->scale) > 1e6 || std::fabs(d->scale) < 1e-6)
    return fail(ZERO_ERR_INVALID, "%s: the magnitude of scale must lie in [1e-6, 1e6]", fn);
  if (d->x_stride < d->hidden || d->x_stride > INT64_C(1) << 36 || d->w_stride < d->hidden ||
      d->w_stride > INT64_C(1) << 36)
    return fail(ZERO_ERR_INVALID, "%s: strides must be at least hidden", fn);
  return ZERO_OK;
}

zero_status check_ptr(const char* fn, const char* what, const void* p, int bytes, bool needed) {
  if (needed && !p) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, bytes)) return fail(ZERO_ERR_ALIGN, "%s: %s is not aligned to %d bytes", fn, what, bytes);
  return ZERO_OK;
}

#define LOSS_TRY(x)                 \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)
#define LOSS_CUDA(x)                                                                                       \
  do {                                                                                                     \
    const cudaError_t e_ = (x);                                                                            \
    if (e_ != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e_)); \
  } while (0)

// What both passes start with: the repacked w, the maps and common arguments
// of the products over x and w.
struct Call {
  const zero_linear_ce_desc& d;
  const Layout at;
  char* ws;
  cudaStream_t s;
  bool bf16;
  const void* w;
  RowsArgs rows = {};
  ProductArgs product = {};

  Call(const zero_linear_ce_desc& d_, const Layout& at_, void* ws_, void* stream, const void* w_)
      : d(d_), at(at_), ws(static_cast<char*>(ws_)), s(static_cast<cudaStream_t>(stream)), bf16(d_.dtype == ZERO_BF16),
        w(w_) {}
  template <class T>
  T* in(int64_t offset) const { return reinterpret_cast<T*>(ws + offset); }

  void set_vec(bool vec) { rows.vec = vec, rows.log_lanes = lanes_for(d.hidden, 32); }
  zero_status begin(const char* fn, const void* x, const void* targets, int32_t* row_list, int32_t* err) {
    rows.targets = targets, rows.id_bytes = d.id_bytes, rows.vocab = static_cast<int32_t>(d.vocab);
    rows.tokens = d.tokens, rows.hidden = d.hidden, rows.rows = row_list, rows.ticket = in<int32_t>(at.ticket);
    rows.err = product.err = err, rows.gave_up = product.gave_up = rows.ticket + 1;
    rows.x = x, rows.x_stride = d.x_stride, rows.xs = in<void>(at.xs), rows.xs_stride = at.xs_stride;
    rows.rows_cap = at.rows_cap, rows.target = in<int32_t>(at.target);
    set_vec(d.hidden % 8 == 0 && d.x_stride % 8 == 0 && aligned_to(x, 16));
    product.count = row_list + d.tokens, product.rows_cap = at.rows_cap;
    product.hidden = static_cast<int32_t>(d.hidden);
    product.bf16 = bf16, product.scale2 = static_cast<float>(d.scale * 1.4426950408889634);
    product.target = rows.target, product.rows = row_list, product.tokens = d.tokens;
    product.pieces = static_cast<int32_t>(at.pieces), product.piece = static_cast<int32_t>(at.columns);
    int pairs = 0;
    static KernelFacts facts;
    const void* k = reinterpret_cast<const void*>(&k_loss_product<kStats>);
    LOSS_CUDA(facts.allow(k, kSmemBytes, kSmemBytes));
    LOSS_CUDA(pairs_of(k, &pairs));
    product.pairs = pairs;
    product.rows_a = d.tokens < kHalfRows ? static_cast<int32_t>(up(std::max<int64_t>(d.tokens, 1), 16)) : kHalfRows;
    return ZERO_OK;
  }
  // rows of `bytes`-wide elements to another stride
  CopyArgs copy_of(const void* from, int64_t from_stride, void* to, int64_t to_stride, int64_t n, int bytes) const {
    const int log_lanes = lanes_for(d.hidden, 32);
    return {from, to, from_stride, to_stride, n, static_cast<int32_t>(d.hidden), log_lanes, bytes / 2,
            ctas_for(n, log_lanes)};
  }
  // w as the bulk copies can take it, and what brings it there
  CopyArgs repack() {
    if (!wants_repack(d, w)) return {};
    const CopyArgs copy = copy_of(w, d.w_stride, in<void>(at.w), at.w_stride, d.vocab, 2);
    w = copy.to;
    return copy;
  }
  // rows of xs and of w, contiguous along the depth; tiles for `columns` of z
  bool maps_of_z(int64_t columns) {
    product.narrow = narrow_columns(at.rows_cap / kTileM, columns, product.pairs);
    const void* xs = in<void>(at.xs);
    return matrix_map(&product.a, xs, bf16, d.hidden, at.rows_cap, at.xs_stride, product.rows_a) &&
           matrix_map(&product.b, w, bf16, d.hidden, d.vocab, at.w_stride, kHalfRows) &&
           matrix_map(&product.b2, w, bf16, d.hidden, d.vocab, at.w_stride, product.narrow / 2);
  }
};

// The device can run the products and nothing is pending.
zero_status ready(const char* fn, int32_t** err) {
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  *err = device_error_word();
  if (!*err) return fail(ZERO_ERR_CUDA, "%s: no device error word", fn);
  return ZERO_OK;
}

int align_of(const void* p, int64_t row_bytes) {
  const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)) | row_bytes;
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 2;
}

Extent by_rows(const char* name, const void* p, int64_t rows, int64_t stride, int64_t hidden) {
  return {name, p, rows, stride * 2, hidden * 2};
}

zero_status forward(const char* fn, const zero_linear_ce_desc* desc, const void* x, const void* w, const void* targets,
                    float* losses, float* lse, float* rest, bool with_rest, int32_t* rows, float* total,
                    void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  NvtxRange range(fn);
  LOSS_TRY(check_desc(fn, desc));
  const zero_linear_ce_desc& d = *desc;
  const bool any = d.tokens > 0;
  LOSS_TRY(check_ptr(fn, "x", x, 2, any));
  LOSS_TRY(check_ptr(fn, "w", w, 2, true));
  LOSS_TRY(check_ptr(fn, "targets", targets, d.id_bytes, any));
  LOSS_TRY(check_ptr(fn, "losses", losses, 4, any));
  LOSS_TRY(check_ptr(fn, "lse", lse, 4, any));
  LOSS_TRY(check_ptr(fn, "rest", rest, 4, any && with_rest));
  LOSS_TRY(check_ptr(fn, "rows", rows, 4, true));
  LOSS_TRY(check_ptr(fn, "total", total, 4, true));
  LOSS_TRY(check_ptr(fn, "workspace", workspace, 256, true));
  const Layout at(d, wants_repack(d, w), false);
  if (workspace_bytes < at.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes,
                at.bytes);
  LOSS_TRY(check_overlaps(fn,
                          {Extent::block("losses", losses, d.tokens * 4), Extent::block("lse", lse, d.tokens * 4),
                           Extent::block("rest", rest, d.tokens * 4), Extent::block("rows", rows, (d.tokens + 1) * 4), Extent::block("total", total, 12),
                           Extent::block("workspace", workspace, at.bytes)},
                          {by_rows("x", x, d.tokens, d.x_stride, d.hidden), by_rows("w", w, d.vocab, d.w_stride, d.hidden),
                           Extent::block("targets", targets, d.tokens * d.id_bytes)}));
  int32_t* err = nullptr;
  LOSS_TRY(ready(fn, &err));
  Call c(d, at, workspace, stream, w);
  LOSS_TRY(c.begin(fn, x, targets, rows, err));
  const CopyArgs repack = c.repack();
  if (d.tokens <= kFewTokens) {
    LOSS_CUDA(launch_gather<kForwardFew>(c.rows, repack, false, c.s));
  } else {
    LOSS_CUDA(launch(&k_loss_rows, 1, kScanThreads, 0, false, c.s, static_cast<const RowsArgs>(c.rows)));
    LOSS_CUDA(launch_gather<kForward>(c.rows, repack, true, c.s));
  }
  if (!c.maps_of_z(d.vocab)) return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
  c.product.columns = static_cast<int32_t>(d.vocab);
  c.product.part = c.in<float2>(at.part), c.product.target_z = c.in<float>(at.target_z);
  LOSS_CUDA(d.hidden > kSegment * kTileK ? launch_product<kStatsLong>(c.product, c.s)
                                         : launch_product<kStats>(c.product, c.s));
  c.rows.narrow = c.product.narrow, c.rows.pairs = c.product.pairs;
  c.rows.part = c.product.part, c.rows.target_z = c.product.target_z;
  c.rows.cta_sums = c.in<float>(at.cta_sums), c.rows.losses = losses, c.rows.lse_out = lse;
  c.rows.rest_out = rest, c.rows.total = total;
  LOSS_CUDA(launch(&k_loss_finish, std::max<int64_t>(1, over(d.tokens, kFinishRows)), kFinishThreads, 0, true, c.s,
                   static_cast<const RowsArgs>(c.rows)));
  return ZERO_OK;
}

zero_status backward(const char* fn, const zero_linear_ce_desc* desc, const void* x, const void* w,
                     const void* targets, const float* lse, const float* rest, bool with_rest, const int32_t* rows,
                     const float* d_loss, int32_t reduction, void* dx, void* dw, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  clear_error();
  NvtxRange range(fn);
  LOSS_TRY(check_desc(fn, desc));
  const zero_linear_ce_desc& d = *desc;
  const bool any = d.tokens > 0;
  if (reduction != ZERO_LOSS_NONE && reduction != ZERO_LOSS_SUM && reduction != ZERO_LOSS_MEAN)
    return fail(ZERO_ERR_INVALID, "%s: unknown reduction", fn);
  const zero_dtype dw_dtype = d.dw_dtype;
  LOSS_TRY(check_ptr(fn, "x", x, 2, any));
  LOSS_TRY(check_ptr(fn, "w", w, 2, true));
  LOSS_TRY(check_ptr(fn, "targets", targets, d.id_bytes, any));
  LOSS_TRY(check_ptr(fn, "lse", lse, 4, any));
  LOSS_TRY(check_ptr(fn, "rest", rest, 4, any && with_rest));
  LOSS_TRY(check_ptr(fn, "rows", rows, 4, true));
  LOSS_TRY(check_ptr(fn, "d_loss", d_loss, 4, any || reduction != ZERO_LOSS_NONE));
  LOSS_TRY(check_ptr(fn, "dx", dx, 2, false));
  LOSS_TRY(check_ptr(fn, "dw", dw, type_bytes(dw_dtype), false));
  LOSS_TRY(check_ptr(fn, "workspace", workspace, 256, true));
  if (!any) dx = nullptr;
  if (!dx && !dw) return ZERO_OK;
  const bool own = own_scales(d, reduction, dx);
  const Layout at(d, wants_repack(d, w), true, own && dw);
  const int64_t need = workspace_of(d, w, true);
  if (workspace_bytes < need)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes, need);
  LOSS_TRY(check_overlaps(fn,
                          {Extent::block("dx", dx, d.tokens * d.hidden * 2),
                           Extent::block("dw", dw, d.vocab * d.hidden * type_bytes(dw_dtype)),
                           Extent::block("workspace", workspace, need)},
                          {by_rows("x", x, d.tokens, d.x_stride, d.hidden), by_rows("w", w, d.vocab, d.w_stride, d.hidden),
                           Extent::block("targets", targets, d.tokens * d.id_bytes),
                           Extent::block("lse", lse, d.tokens * 4), Extent::block("rest", rest, d.tokens * 4),
                           Extent::block("rows", rows, (d.tokens + 1) * 4),
                           Extent::block("d_loss", d_loss, reduction == ZERO_LOSS_NONE ? d.tokens * 4 : 4)}));
  int32_t* err = nullptr;
  LOSS_TRY(ready(fn, &err));
  Call c(d, at, workspace, stream, w);
  LOSS_TRY(c.begin(fn, x, targets, const_cast<int32_t*>(rows), err));
  c.rows.lse = lse, c.rows.d = d_loss, c.rows.reduction = reduction, c.rows.scale = d.scale;
  c.rows.scales = c.in<Scales>(at.scales), c.rows.lse2 = c.in<float>(at.lse2), c.rows.row_mul = c.in<float>(at.row_mul);
  c.rows.rest = rest, c.rows.row_rest = c.in<float>(at.row_rest), c.rows.dx = dx;
  if (own) c.rows.row_alpha = c.in<float>(at.row_alpha), c.rows.row_own = dw ? c.in<float>(at.row_own) : nullptr;
  c.set_vec(c.rows.vec && aligned_to(dx, 16));
  const bool own_gradients = reduction == ZERO_LOSS_NONE;
  if (own_gradients)
    LOSS_CUDA(launch(&k_loss_scales, 1, kScanThreads, 0, false, c.s, static_cast<const RowsArgs>(c.rows)));
  LOSS_CUDA(launch_gather<kBackward>(c.rows, c.repack(), own_gradients, c.s));
  CopyArgs copy = {};  // of dw, after a piece's products
  if (!c.maps_of_z(std::min(at.columns, d.vocab))) return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
  ProductArgs z = c.product;
  z.lse2 = c.rows.lse2, z.row_mul = c.rows.row_mul, z.row_own = c.rows.row_own, z.row_alpha = c.rows.row_alpha;
  z.scales = c.rows.scales, z.rest = rest ? c.rows.row_rest : nullptr;
  z.dz = c.in<void>(at.dz), z.dz_stride = at.columns;
  z.terms = dw ? at.terms : 1;
  for (int64_t first = 0; first < d.vocab; first += at.columns) {
    const int64_t columns = std::min(at.columns, d.vocab - first);
    z.first = static_cast<int32_t>(first), z.columns = static_cast<int32_t>(columns);
    LOSS_CUDA(launch_product<kProbs>(z, c.s));
    ProductArgs p = z;
    p.sums = c.in<float>(at.sums), p.sums_stride = at.sums_stride, p.add = first > 0, p.direct = at.whole;
    p.dx = {dx, d.hidden, 0, d.dtype, align_of(dx, d.hidden * 2)};
    // rows that start anywhere are written to a padded copy first: single columns
    // from a row a thread took 77 us, copy and all 24 (5003 x 1001 fp16)
    if (dw && at.whole)
      p.dw = {dw, d.hidden, first, dw_dtype, align_of(dw, d.hidden * type_bytes(dw_dtype))};
    else if (dw)
      p.dw = {c.in<void>(at.dw), at.sums_stride, 0, dw_dtype, align_of(c.in<void>(at.dw), at.sums_stride * type_bytes(dw_dtype))};
    if (!matrix_map(&p.a, z.dz, c.bf16, columns, at.all_rows, at.columns, kHalfRows) ||
        !matrix_map(&p.b, c.w, c.bf16, d.hidden, d.vocab, at.w_stride, kTileK) ||
        !matrix_map(&p.a2, z.dz, c.bf16, columns, at.dz_rows, at.columns, kTileK) ||
        !matrix_map(&p.b2, c.in<void>(at.xs), c.bf16, d.hidden, at.rows_cap, at.xs_stride, kTileK))
      return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
    LOSS_CUDA(z.terms > 1 ? launch_product<kGradsLong>(p, c.s) : launch_product<kGrads>(p, c.s));
    if (dw && !at.whole) {
      const int bytes = type_bytes(dw_dtype);
      copy = c.copy_of(p.dw.p, p.dw.stride, static_cast<char*>(dw) + first * d.hidden * bytes, d.hidden, columns, bytes);
      if (first + at.columns < d.vocab)
        LOSS_CUDA(launch(&k_loss_copy, copy.ctas, kGatherThreads, 0, true, c.s, static_cast<const CopyArgs>(copy)));
    }
  }
  // dw alone as well: it is the last to look whether a wait gave up
  JoinArgs j = {};
  j.rows = rows, j.tokens = d.tokens, j.sums = c.in<float>(at.sums), j.sums_stride = at.sums_stride;
  j.scales = c.rows.scales, j.row_alpha = c.rows.row_alpha, j.gave_up = c.rows.gave_up;
  j.dx = dx, j.dw = dw, j.dw_size = d.vocab * d.hidden, j.dw_type = dw_dtype;
  j.hidden = static_cast<int32_t>(d.hidden), j.piece = c.product.piece, j.pieces = c.product.pieces;
  j.pairs = c.product.pairs, j.direct = at.whole, j.vec = at.whole && aligned_to(dx, 16);
  j.log_lanes = lanes_for(d.hidden, 8);
  const int64_t join_ctas = dx ? ctas_for(d.tokens, j.log_lanes) : copy.ctas ? 0 : kSMs;
  LOSS_CUDA(launch(c.bf16 ? &k_loss_join<__nv_bfloat16> : &k_loss_join<__half>, copy.ctas + join_ctas, kGatherThreads, 0,
                   true, c.s, static_cast<const JoinArgs>(j), static_cast<const CopyArgs>(copy)));
  return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_linear_cross_entropy_workspace_bytes(const zero_linear_ce_desc* desc, const void* w,
                                                                 int32_t backward, int64_t* bytes) {
  const char* fn = "zero_linear_cross_entropy_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  LOSS_TRY(check_desc(fn, desc));
  *bytes = workspace_of(*desc, w, backward != 0);
  return ZERO_OK;
}

extern "C" zero_status zero_linear_cross_entropy(const zero_linear_ce_desc* desc, const void* x, const void* w,
                                                 const void* targets, float* losses, float* lse, int32_t* rows,
                                                 float* total, void* workspace, int64_t workspace_bytes,
                                                 void* stream) {
  return forward("zero_linear_cross_entropy", desc, x, w, targets, losses, lse, nullptr, false, rows, total, workspace,
                 workspace_bytes, stream);
}

extern "C" zero_status zero_linear_cross_entropy_rest(const zero_linear_ce_desc* desc, const void* x, const void* w,
                                                      const void* targets, float* losses, float* lse, float* rest,
                                                      int32_t* rows, float* total, void* workspace,
                                                      int64_t workspace_bytes, void* stream) {
  return forward("zero_linear_cross_entropy_rest", desc, x, w, targets, losses, lse, rest, true, rows, total, workspace,
                 workspace_bytes, stream);
}

extern "C" zero_status zero_linear_cross_entropy_backward(const zero_linear_ce_desc* desc, const void* x,
                                                          const void* w, const void* targets, const float* lse,
                                                          const int32_t* rows, const float* d_loss, int32_t reduction,
                                                          void* dx, void* dw, void* workspace,
                                                          int64_t workspace_bytes, void* stream) {
  return backward("zero_linear_cross_entropy_backward", desc, x, w, targets, lse, nullptr, false, rows, d_loss,
                  reduction, dx, dw, workspace, workspace_bytes, stream);
}

extern "C" zero_status zero_linear_cross_entropy_rest_backward(const zero_linear_ce_desc* desc, const void* x,
                                                               const void* w, const void* targets, const float* lse,
                                                               const float* rest, const int32_t* rows,
                                                               const float* d_loss, int32_t reduction, void* dx,
                                                               void* dw, void* workspace, int64_t workspace_bytes,
                                                               void* stream) {
  return backward("zero_linear_cross_entropy_rest_backward", desc, x, w, targets, lse, rest, true, rows, d_loss,
                  reduction, dx, dw, workspace, workspace_bytes, stream);
}
