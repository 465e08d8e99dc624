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
// Four products of one kernel (k_loss_product) make up the two passes:
//   kStats  tiles of z, of which only every row's maximum and sum of
//           exponentials leave the SM; joined by k_loss_finish
//   kProbs  tiles of z again, to dz in 16 bits, a piece of the vocabulary at a
//           time (kPieceBytes)
//   kDx     dz w, summed over the pieces in binary32
//   kDw     dz^T x, the piece's rows of dw
// The second forming of z is a quarter of the operations: the price of keeping
// no logits between the passes.
#include <cuda.h>
#include <cuda_runtime.h>
#include <inttypes.h>

#include <algorithm>
#include <cmath>

#include "zero_capi_util.h"
#include "zero_internal.h"
#include "zero_rows.cuh"
#include "zero_tensor_core.cuh"

namespace zero {
namespace {

constexpr int kTileM = 256, kTileN = 256;  // of a pair of CTAs; each holds half of both operands' rows
constexpr int kTileK = 64;                 // 128 bytes of 16-bit data: one swizzled row
constexpr int kHalfRows = 128;
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalfRows * kTileK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kThreads = 192;  // copies, products, four warps of epilogue
constexpr int kAccumulators = 2;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes;
constexpr int64_t kPieceBytes = INT64_C(512) << 20;  // of dz in memory at a time
constexpr int kGroupM = 8;  // row tiles that run through the column tiles together (their operands stay in L2)
constexpr int kPairsMost = kSMs / 2;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Product { kStats, kProbs, kDx, kDw };

// What the host does not know: the kept rows, and what scales them.
struct Scales {
  float mul;    // of dz before it is rounded, a power of two: largest |dz| below 2^14
  float alpha;  // of the products, scale / mul
  float g;      // d_loss as one number (sum, mean)
};

struct ProductArgs {
  CUtensorMap a, b;
  const int32_t* count;  // kept rows n
  int64_t rows_cap;      // n rounded up to whole tiles at most
  int32_t vocab, hidden;
  int32_t first;         // the piece's first column of z
  int32_t columns;       // of the piece
  int32_t piece;         // columns of a whole piece
  int32_t bf16;
  int32_t* err;
  // kStats, kProbs
  float scale2;          // scale * log2(e)
  const int32_t* target;
  float2* part;          // [column tiles][rows_cap]: maximum and sum, base 2
  float* target_z;       // base 2
  const float* lse2;
  const float* row_mul;
  void* dz;              // [rows_cap][dz_stride]
  int64_t dz_stride;
  // kDx, kDw
  const Scales* scales;
  const int32_t* rows;   // kept row -> token
  int64_t tokens;
  void* out;
  int32_t out_type, out_align;
  float* sums;           // kDx: [splits][n rounded up][sums_stride]
  int64_t sums_stride;
  int32_t add, pieces, pairs;
};

__host__ __device__ __forceinline__ int64_t up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
__host__ __device__ __forceinline__ int64_t over(int64_t n, int64_t unit) { return (n + unit - 1) / unit; }

// How many parts kDx's sum over the vocabulary is cut into, so that few row
// tiles still fill the SMs (their sums are joined by k_loss_join).
__host__ __device__ __forceinline__ int split_of(int64_t tiles, int64_t depth, int pairs) {
  if (tiles < 1 || tiles * 2 > pairs) return 1;
  const int64_t most = over(depth, 4 * kTileK);
  const int64_t s = pairs / tiles;
  return static_cast<int>(s < most ? s : most < 1 ? 1 : most);
}

// The tiles of a product and their order.
template <int KIND>
struct Tiles {
  int m_tiles, n_tiles, splits, depth_blocks;
  int64_t total;
  __device__ __forceinline__ Tiles(const ProductArgs& a, int n) {
    const int rows = KIND == kDw ? a.columns : n;
    const int cols = KIND == kDx || KIND == kDw ? a.hidden : a.columns;
    const int depth = KIND == kDx ? a.columns : KIND == kDw ? n : a.hidden;
    m_tiles = static_cast<int>(over(rows, kTileM));
    n_tiles = static_cast<int>(over(cols, kTileN));
    depth_blocks = static_cast<int>(over(depth, kTileK));
    splits = KIND == kDx ? split_of(static_cast<int64_t>(m_tiles) * n_tiles, a.piece, a.pairs) : 1;
    total = static_cast<int64_t>(m_tiles) * n_tiles * splits;
  }
  __device__ __forceinline__ void at(int64_t t, int& m, int& n, int& s) const {
    const int64_t plane = static_cast<int64_t>(m_tiles) * n_tiles;
    s = static_cast<int>(t / plane);
    t -= s * plane;
    const int64_t group = static_cast<int64_t>(kGroupM) * n_tiles;
    const int m0 = static_cast<int>(t / group) * kGroupM;
    const int size = min(kGroupM, m_tiles - m0);
    t -= t / group * group;
    n = static_cast<int>(t / size);
    m = m0 + static_cast<int>(t % size);
  }
  __device__ __forceinline__ void depth(int s, int& k0, int& k1) const {
    k0 = static_cast<int>(static_cast<int64_t>(depth_blocks) * s / splits);
    k1 = static_cast<int>(static_cast<int64_t>(depth_blocks) * (s + 1) / splits);
  }
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

// A tile's epilogue for one row: 256 columns, 32 at a time, from tensor memory.
template <int KIND>
struct Epilogue {
  const ProductArgs& a;
  int n;            // kept rows
  int64_t row;      // of the product
  int m, col, split, k_blocks;

  // maximum and sum of exponentials so far
  float top = -INFINITY, sum = 0.f;
  int target = -1;
  float lse2 = 0.f, mul = 0.f;
  float alpha = 0.f;
  int64_t token = -1;
  bool direct = true;
  int64_t sums_rows = 0;

  __device__ __forceinline__ Epilogue(const ProductArgs& a_, int n_, const Tiles<KIND>& t, int m_, int nt, int split_,
                                      int row_in_tile)
      : a(a_), n(n_), m(m_), split(split_) {
    row = static_cast<int64_t>(m_) * kTileM + row_in_tile;
    col = nt * kTileN;
    const bool live = KIND == kDw ? row < a.columns : row < n;
    if constexpr (KIND == kStats || KIND == kProbs) {
      if (live) target = a.target[row] - a.first;
    }
    if constexpr (KIND == kProbs) {
      if (live) lse2 = a.lse2[row], mul = a.row_mul[row];
    }
    if constexpr (KIND == kDx) {
      direct = a.pieces == 1 && t.splits == 1;
      sums_rows = up(n, kTileM);
      if (live) token = a.rows[row];
      if (token >= a.tokens) token = -1;
      alpha = a.scales->alpha;
    }
    if constexpr (KIND == kDw) {
      if (live) token = a.first + row;
      alpha = a.scales->alpha;
    }
    (void)live;
  }

  __device__ __forceinline__ void take(const uint32_t (&w)[32], int c0, bool zero) {
    const int c = col + c0;
    if constexpr (KIND == kStats) {
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = __uint_as_float(w[i]) * a.scale2;
      if (c + 32 > a.columns) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i >= a.columns) t[i] = -INFINITY;
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
      const int rel = target - c;
      if (__any_sync(kFull, rel >= 0 && rel < 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (rel == i) a.target_z[row] = t[i];
      }
    } else if constexpr (KIND == kProbs) {
      float p[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i] = tc::exp2_of(fmaf(__uint_as_float(w[i]), a.scale2, -lse2));
      const int rel = target - c;
      if (__any_sync(kFull, rel >= 0 && rel < 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (rel == i) p[i] -= 1.f;
      }
      if (row < n) {
#pragma unroll
        for (int i = 0; i < 32; ++i) p[i] *= mul;
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) p[i] = 0.f;
      }
      if (a.bf16)
        store32(static_cast<__nv_bfloat16*>(a.dz) + row * a.dz_stride + c, p, 32, 32);
      else
        store32(static_cast<__half*>(a.dz) + row * a.dz_stride + c, p, 32, 32);
    } else {
      const int left = a.hidden - c;
      if (left <= 0) return;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = zero ? 0.f : __uint_as_float(w[i]);
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
      const int64_t at = token * a.hidden + c;
      if (a.out_type == ZERO_FP32)
        store32(static_cast<float*>(a.out) + at, v, left, a.out_align);
      else if (a.out_type == ZERO_BF16)
        store32(static_cast<__nv_bfloat16*>(a.out) + at, v, left, a.out_align);
      else
        store32(static_cast<__half*>(a.out) + at, v, left, a.out_align);
    }
  }

  __device__ __forceinline__ void done() {
    if constexpr (KIND == kStats) a.part[static_cast<int64_t>(col / kTileN) * a.rows_cap + row] = make_float2(top, sum);
  }
};

// A persistent pair of CTAs a tile of 256 x 256: one thread of each CTA copies
// its half of the operands' blocks into a ring of kStages, one thread of the
// leading CTA issues the products of both, and four warps of each CTA work on
// its half of a finished tile in tensor memory while the next one is formed in
// the other accumulator.
template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_loss_product(const __grid_constant__ ProductArgs a) {
  extern __shared__ char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kAccumulators + 1];
  __shared__ uint32_t tmem_slot;
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
    for (int s = 0; s < kStages; ++s) tc::bar_init(full(s), 1), tc::bar_init(empty(s), 1);
    for (int s = 0; s < kAccumulators; ++s) tc::bar_init(acc_full(s), 1), tc::bar_init(acc_empty(s), 8);
    tc::bar_init(drained, 1);
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_of(&tmem_slot), kAccumulators * kTileN);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_previous();

  const int n = *a.count;
  const Tiles<KIND> tiles(a, n);
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  constexpr bool kAByM = KIND == kDw, kBByN = KIND == kDx || KIND == kDw;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    Ring<kStages> ring;
    int64_t issued = 0;
    for (int64_t t = first; t < tiles.total && ok; t += step) {
      int m, nt, s, k0, k1;
      tiles.at(t, m, nt, s);
      tiles.depth(s, k0, k1);
      const int row = m * kTileM + static_cast<int>(rank) * kHalfRows, col = nt * kTileN + static_cast<int>(rank) * kHalfRows;
      for (int k = k0; k < k1; ++k) {
        ok = tc::bar_wait(empty(ring.slot), ring.phase ^ 1);
        if (!ok) break;
        const uint32_t dst = base + ring.slot * kStageBytes;
        const uint32_t bar = tc::in_cta(full(ring.slot), 0);
        if (rank == 0) tc::bar_expect(full(ring.slot), 2 * kStageBytes);
        if constexpr (kAByM) {
          tc::load_box(dst, &a.a, row, k * kTileK, bar);
          tc::load_box(dst + kOperandBytes / 2, &a.a, row + 64, k * kTileK, bar);
        } else {
          tc::load_box(dst, &a.a, k * kTileK, row, bar);
        }
        if constexpr (kBByN) {
          const int depth = k * kTileK + (KIND == kDx ? a.first : 0);
          tc::load_box(dst + kOperandBytes, &a.b, col, depth, bar);
          tc::load_box(dst + kOperandBytes + kOperandBytes / 2, &a.b, col + 64, depth, bar);
        } else {
          tc::load_box(dst + kOperandBytes, &a.b, k * kTileK, a.first + col, bar);
        }
        ++issued;
        ring.next();
      }
    }
    if (!ok) {
      // given up: wait for the copies of both CTAs before the memory goes
      atomicExch(a.err, 1);
      if (rank == 0)
        for (int64_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
          tc::bar_wait(full(static_cast<int>(j % kStages)), static_cast<uint32_t>(j / kStages) & 1);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    const uint32_t instr = tc::instruction(a.bf16 != 0, kAByM, kBByN, kTileM, kTileN);
    constexpr uint32_t kLead = kOperandBytes / 2;
    Ring<kStages> ring;
    Ring<kAccumulators> acc;
    for (int64_t t = first; t < tiles.total && ok; t += step) {
      int m, nt, s, k0, k1;
      tiles.at(t, m, nt, s);
      tiles.depth(s, k0, k1);
      ok = tc::bar_wait(acc_empty(acc.slot), acc.phase ^ 1);
      if (!ok) break;
      tc::fence_after();
      const uint32_t d = tmem + acc.slot * kTileN;
      for (int k = k0; k < k1; ++k) {
        ok = tc::bar_wait(full(ring.slot), ring.phase);
        if (!ok) break;
        tc::fence_after();
        const uint32_t at_a = base + ring.slot * kStageBytes, at_b = at_a + kOperandBytes;
        const uint64_t da = tc::operand(at_a, kAByM ? kLead : 16, 1024);
        const uint64_t db = tc::operand(at_b, kBByN ? kLead : 16, 1024);
#pragma unroll
        for (int i = 0; i < kTileK / 16; ++i) {
          // 16 deep: 32 bytes along a row, or 16 rows of 128 bytes
          const uint64_t step_a = (kAByM ? 2048 : 32) >> 4, step_b = (kBByN ? 2048 : 32) >> 4;
          tc::mma(d, da + i * step_a, db + i * step_b, instr, k > k0 || i > 0);
        }
        tc::commit(empty(ring.slot));
        ring.next();
      }
      if (!ok) break;
      tc::commit(acc_full(acc.slot));
      acc.next();
    }
    if (!ok) {
      atomicExch(a.err, 1);
      tc::commit(drained);
      tc::bar_wait(drained, 0);
    }
  } else if (warp >= 2) {
    Ring<kAccumulators> acc;
    const int quarter = warp & 3;  // the rows of tensor memory that this warp may read
    for (int64_t t = first; t < tiles.total && ok; t += step) {
      int m, nt, s, k0, k1;
      tiles.at(t, m, nt, s);
      tiles.depth(s, k0, k1);
      Epilogue<KIND> e(a, n, tiles, m, nt, s, static_cast<int>(rank) * kHalfRows + quarter * 32 + lane);
      ok = tc::bar_wait(acc_full(acc.slot), acc.phase);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      tc::fence_after();
      const uint32_t d = tmem + acc.slot * kTileN + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int c = 0; c < kTileN; c += 32) {
        uint32_t w[32];
        tc::tmem_load(d + c, w);
        tc::tmem_wait_load();
        e.take(w, c, k0 == k1);
      }
      e.done();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive_cluster(tc::in_cta(acc_empty(acc.slot), 0));
      acc.next();
    }
    if (!ok && lane == 0) atomicExch(a.err, 1);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // no CTA leaves while the other may still write to it
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
  // gathering
  const void* x;
  int64_t x_stride, xs_stride, rows_cap;
  void* xs;
  int32_t* target;
  int32_t vec;
  // gradients
  const float* lse;
  const float* d;
  int32_t reduction;
  double scale;
  Scales* scales;
  float *lse2, *row_mul;
  void* dx;
  int32_t dx_bytes;
  // losses
  const float2* part;
  const float* target_z;
  int32_t column_tiles;
  float *losses, *lse_out, *total;
};

__device__ __forceinline__ int load_target(const RowsArgs& a, int64_t t) {
  if (a.id_bytes == 4) {
    const int v = static_cast<const int*>(a.targets)[t];
    return v >= 0 && v < a.vocab ? v : -1;
  }
  const long long v = static_cast<const long long*>(a.targets)[t];
  return v >= 0 && v < a.vocab ? static_cast<int>(v) : -1;
}

// The kept tokens, in order: one CTA, a token's target each round and thread.
constexpr int kScanThreads = 1024, kScanEach = 4;
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
#pragma unroll
    for (int i = 0; i < kScanEach; ++i) {
      const int64_t t = w0 + 32 * i + lane;
      kept[i] = t < a.tokens && load_target(a, t) >= 0;
    }
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
// brings the largest to [2^13, 2^14), so that neither rounding to 16 bits nor
// fp16's range costs small probabilities.
__global__ void __launch_bounds__(kScanThreads) k_loss_scales(const RowsArgs a) {
  __shared__ float most[32];
  let_next_start();
  const int n = a.rows[a.tokens];
  float g = 0.f, top = 0.f;
  if (a.reduction == ZERO_LOSS_NONE) {
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
      const int t = a.rows[i];
      if (t >= 0 && t < a.tokens) top = fmaxf(top, fabsf(a.d[t]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = top;
    __syncthreads();
    top = most[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  } else {
    g = *a.d;
    if (a.reduction == ZERO_LOSS_MEAN) g = g / static_cast<float>(max(n, 1));
    top = fabsf(g);
  }
  if (threadIdx.x == 0) {
    int e = 14;
    if (!(top <= 3.4e38f))
      e = 127;  // infinite or NaN: the results are, too
    else if (top > 0.f)
      frexpf(top, &e);
    e = max(e, -100);
    *a.scales = {ldexpf(1.f, 14 - e), static_cast<float>(ldexp(a.scale, e - 14)), g};
  }
}

// The kept rows copied together, zeros up to a whole tile; their targets (and,
// for the gradients, what scales them); left-out rows of dx.
constexpr int kGatherThreads = 256;
template <class W, bool BACKWARD>
__global__ void __launch_bounds__(kGatherThreads) k_loss_gather(const RowsArgs a) {
  let_next_start();
  wait_for_previous();
  const int n = a.rows[a.tokens];
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kGatherThreads / 32);
  const int words = static_cast<int>(a.hidden * 2 / sizeof(W));
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kGatherThreads / 32) + (threadIdx.x >> 5); i < a.rows_cap;
       i += warps) {
    if (i < up(n, kTileM)) {
      const int t = i < n ? a.rows[i] : -1;
      W* to = reinterpret_cast<W*>(static_cast<char*>(a.xs) + i * a.xs_stride * 2);
      if (t >= 0 && t < a.tokens) {
        const W* from = reinterpret_cast<const W*>(static_cast<const char*>(a.x) + t * a.x_stride * 2);
#pragma unroll 4
        for (int c = lane; c < words; c += 32) to[c] = from[c];
        if (lane == 0) {
          const int target = load_target(a, t);
          a.target[i] = target;
          if constexpr (BACKWARD) {
            a.lse2[i] = a.lse[t] * kLog2e;
            const float g = a.reduction == ZERO_LOSS_NONE ? a.d[t] : a.scales->g;
            a.row_mul[i] = target < 0 ? 0.f : g * a.scales->mul;
          }
        }
      } else {
        for (int c = lane; c < words; c += 32) to[c] = W();
        if (lane == 0) {
          a.target[i] = -1;
          if constexpr (BACKWARD) a.lse2[i] = 0.f, a.row_mul[i] = 0.f;
        }
      }
    }
    if constexpr (BACKWARD) {
      if (a.dx && i < a.tokens && load_target(a, i) < 0) {
        W* to = reinterpret_cast<W*>(static_cast<char*>(a.dx) + i * a.hidden * 2);
        for (int c = lane; c < words; c += 32) to[c] = W();
      }
    }
  }
}

// w at a stride that the bulk copies can take.
__global__ void __launch_bounds__(kGatherThreads) k_loss_repack(const uint16_t* __restrict__ w, int64_t stride,
                                                                uint16_t* __restrict__ to, int64_t to_stride,
                                                                int64_t rows, int hidden) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kGatherThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kGatherThreads / 32) + (threadIdx.x >> 5); i < rows; i += warps)
#pragma unroll 8
    for (int c = lane; c < hidden; c += 32) to[i * to_stride + c] = w[i * stride + c];
}

// Every kept row's statistics joined over the column tiles, eight threads a
// row; the CTA that is last adds the losses up, in one order.
constexpr int kFinishRows = 32, kFinishThreads = 256;
__global__ void __launch_bounds__(kFinishThreads) k_loss_finish(const RowsArgs a) {
  __shared__ float2 part[kFinishThreads / kFinishRows][kFinishRows];
  __shared__ float sums[kFinishThreads / 32];
  __shared__ bool last;
  wait_for_previous();
  const int n = a.rows[a.tokens];
  const int r = threadIdx.x % kFinishRows, g = threadIdx.x / kFinishRows;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kFinishRows + r;
  float top = -INFINITY, sum = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int v = g; v < a.column_tiles; v += kFinishThreads / kFinishRows) {
      const float2 p = a.part[v * a.rows_cap + i];
      const float most = fmaxf(top, p.x), at = most == -INFINITY ? 0.f : most;
      sum = sum * exp2f(top - at) + p.y * exp2f(p.x - at);
      top = most;
    }
  }
  part[g][r] = make_float2(top, sum);
  __syncthreads();
  if (g == 0) {
    for (int k = 1; k < kFinishThreads / kFinishRows; ++k) {
      const float2 p = part[k][r];
      const float most = fmaxf(top, p.x), at = most == -INFINITY ? 0.f : most;
      sum = sum * exp2f(top - at) + p.y * exp2f(p.x - at);
      top = most;
    }
    if (i < n) {
      const int t = a.rows[i];
      const float lse2 = top + log2f(sum);
      a.lse_out[t] = lse2 * kLn2;
      a.losses[t] = (lse2 - a.target_z[i]) * kLn2;
    }
    if (i < a.tokens && load_target(a, i) < 0) a.lse_out[i] = 0.f, a.losses[i] = 0.f;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // a thread's sum with what its additions lose
  float s = 0.f, lost = 0.f;
  for (int64_t t = threadIdx.x; t < a.tokens; t += kFinishThreads) {
    const float v = __ldcg(a.losses + t), next = s + v;
    lost += fabsf(s) >= fabsf(v) ? (s - next) + v : (v - next) + s;
    s = next;
  }
  if (isfinite(s)) s += lost;
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

// dx from its binary32 sums, where there is more than one part.
struct JoinArgs {
  const int32_t* rows;
  int64_t tokens;
  const float* sums;
  int64_t sums_stride;
  const Scales* scales;
  void* dx;
  int32_t hidden, type, piece, pieces, pairs;
};
__global__ void __launch_bounds__(kGatherThreads) k_loss_join(const JoinArgs a) {
  wait_for_previous();
  const int n = a.rows[a.tokens];
  const int64_t tiles = over(n, kTileM) * over(a.hidden, kTileN);
  const int splits = split_of(tiles, a.piece, a.pairs);
  if (splits == 1 && a.pieces == 1) return;
  const float alpha = a.scales->alpha;
  const int64_t part = up(n, kTileM) * a.sums_stride;
  const int64_t all = static_cast<int64_t>(n) * a.hidden;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kGatherThreads + threadIdx.x; e < all;
       e += static_cast<int64_t>(gridDim.x) * kGatherThreads) {
    const int64_t i = e / a.hidden, c = e - i * a.hidden;
    const float* p = a.sums + i * a.sums_stride + c;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += p[k * part];
    const int64_t t = a.rows[i];
    if (t >= 0 && t < a.tokens) store_any(a.dx, t * a.hidden + c, a.type, s * alpha);
  }
}

// ---------------------------------------------------------------------------
// host

// Where a call's scratch lies.
struct Layout {
  int64_t rows_cap, column_tiles, columns, pieces, xs_stride, w_stride, sums_stride;
  int64_t xs, w, part, target_z, target, ticket, lse2, row_mul, scales, dz, sums, bytes;

  Layout(const zero_linear_ce_desc& d, bool repack, bool backward, bool want_dx) {
    rows_cap = up(std::max<int64_t>(d.tokens, 1), kTileM);
    column_tiles = over(d.vocab, kTileN);
    columns = up(d.vocab, kTileN);
    if (backward) columns = std::min(columns, std::max<int64_t>(kTileN, kPieceBytes / 2 / rows_cap / kTileN * kTileN));
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
    ticket = take(4);
    part = take(backward ? 0 : column_tiles * rows_cap * 8);
    target_z = take(backward ? 0 : rows_cap * 4);
    lse2 = take(backward ? rows_cap * 4 : 0);
    row_mul = take(backward ? rows_cap * 4 : 0);
    scales = take(sizeof(Scales));
    dz = take(backward ? rows_cap * columns * 2 : 0);
    // as many rows as there are tokens, or the parts of few
    const int64_t split_rows = static_cast<int64_t>(kPairsMost) * kTileM;
    sums = take(backward && want_dx
                    ? (pieces > 1 ? std::max(split_rows, rows_cap) : split_rows) * sums_stride * 4
                    : 0);
    bytes = at;
  }
};

bool wants_repack(const zero_linear_ce_desc& d, const void* w) {
  return d.w_stride % 8 != 0 || !aligned_to(w, 16);
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

cudaError_t launch_gather(const RowsArgs& a, bool backward, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(over(a.rows_cap, kGatherThreads / 32), kSMs * 8);
  if (a.vec)
    return backward ? launch(&k_loss_gather<uint4, true>, grid, kGatherThreads, 0, true, s, a)
                    : launch(&k_loss_gather<uint4, false>, grid, kGatherThreads, 0, true, s, a);
  return backward ? launch(&k_loss_gather<uint16_t, true>, grid, kGatherThreads, 0, true, s, a)
                  : launch(&k_loss_gather<uint16_t, false>, grid, kGatherThreads, 0, true, s, a);
}

zero_status check_desc(const char* fn, const zero_linear_ce_desc* d) {
  if (!d) return fail(ZERO_ERR_INVALID, "%s: desc is NULL", fn);
  if (d->tokens < 0 || d->tokens > 1 << 24)
    return fail(ZERO_ERR_INVALID, "%s: tokens must lie in [0, 2^24]", fn);
  if (d->hidden < 1 || d->hidden > 1 << 20) return fail(ZERO_ERR_INVALID, "%s: hidden must lie in [1, 2^20]", fn);
  if (d->vocab < 1 || d->vocab > 1 << 28) return fail(ZERO_ERR_INVALID, "%s: vocab must lie in [1, 2^28]", fn);
  if (d->dtype != ZERO_FP16 && d->dtype != ZERO_BF16)
    return fail(ZERO_ERR_INVALID, "%s: dtype must be ZERO_FP16 or ZERO_BF16", fn);
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

  zero_status begin(const char* fn, const void* x, const void* targets, int32_t* row_list, int32_t* err) {
    rows.targets = targets, rows.id_bytes = d.id_bytes, rows.vocab = static_cast<int32_t>(d.vocab);
    rows.tokens = d.tokens, rows.hidden = d.hidden, rows.rows = row_list, rows.ticket = in<int32_t>(at.ticket);
    rows.x = x, rows.x_stride = d.x_stride, rows.xs = in<void>(at.xs), rows.xs_stride = at.xs_stride;
    rows.rows_cap = at.rows_cap, rows.target = in<int32_t>(at.target);
    rows.vec = d.hidden % 8 == 0 && d.x_stride % 8 == 0 && aligned_to(x, 16);
    product.count = row_list + d.tokens, product.rows_cap = at.rows_cap;
    product.vocab = static_cast<int32_t>(d.vocab), product.hidden = static_cast<int32_t>(d.hidden);
    product.bf16 = bf16, product.err = err, product.scale2 = static_cast<float>(d.scale * 1.4426950408889634);
    product.target = rows.target, product.rows = row_list, product.tokens = d.tokens;
    product.pieces = static_cast<int32_t>(at.pieces), product.piece = static_cast<int32_t>(at.columns);
    int pairs = 0;
    static KernelFacts facts;
    const void* k = reinterpret_cast<const void*>(&k_loss_product<kStats>);
    LOSS_CUDA(facts.allow(k, kSmemBytes, kSmemBytes));
    LOSS_CUDA(pairs_of(k, &pairs));
    product.pairs = pairs;
    return ZERO_OK;
  }
  zero_status repack(const char* fn) {
    if (!wants_repack(d, w)) return ZERO_OK;
    uint16_t* to = in<uint16_t>(at.w);
    LOSS_CUDA(launch(&k_loss_repack, std::min<int64_t>(over(d.vocab, kGatherThreads / 32), kSMs * 8), kGatherThreads, 0,
                     true, s, static_cast<const uint16_t*>(w), d.w_stride, to, at.w_stride, d.vocab,
                     static_cast<int>(d.hidden)));
    w = to;
    return ZERO_OK;
  }
  // rows of xs and of w, contiguous along the depth
  bool maps_of_z() {
    return matrix_map(&product.a, in<void>(at.xs), bf16, d.hidden, at.rows_cap, at.xs_stride, kHalfRows) &&
           matrix_map(&product.b, w, bf16, d.hidden, d.vocab, at.w_stride, kHalfRows);
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

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_linear_cross_entropy_workspace_bytes(const zero_linear_ce_desc* desc, const void* w,
                                                                 int32_t backward, int64_t* bytes) {
  const char* fn = "zero_linear_cross_entropy_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  LOSS_TRY(check_desc(fn, desc));
  *bytes = Layout(*desc, wants_repack(*desc, w), backward != 0, true).bytes;
  return ZERO_OK;
}

extern "C" zero_status zero_linear_cross_entropy(const zero_linear_ce_desc* desc, const void* x, const void* w,
                                                 const void* targets, float* losses, float* lse, int32_t* rows,
                                                 float* total, void* workspace, int64_t workspace_bytes,
                                                 void* stream) {
  const char* fn = "zero_linear_cross_entropy";
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
  LOSS_TRY(check_ptr(fn, "rows", rows, 4, true));
  LOSS_TRY(check_ptr(fn, "total", total, 4, true));
  LOSS_TRY(check_ptr(fn, "workspace", workspace, 256, true));
  const Layout at(d, wants_repack(d, w), false, false);
  if (workspace_bytes < at.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes,
                at.bytes);
  LOSS_TRY(check_overlaps(fn,
                          {Extent::block("losses", losses, d.tokens * 4), Extent::block("lse", lse, d.tokens * 4),
                           Extent::block("rows", rows, (d.tokens + 1) * 4), Extent::block("total", total, 12),
                           Extent::block("workspace", workspace, at.bytes)},
                          {by_rows("x", x, d.tokens, d.x_stride, d.hidden), by_rows("w", w, d.vocab, d.w_stride, d.hidden),
                           Extent::block("targets", targets, d.tokens * d.id_bytes)}));
  int32_t* err = nullptr;
  LOSS_TRY(ready(fn, &err));
  Call c(d, at, workspace, stream, w);
  LOSS_TRY(c.begin(fn, x, targets, rows, err));
  LOSS_CUDA(launch(&k_loss_rows, 1, kScanThreads, 0, false, c.s, static_cast<const RowsArgs>(c.rows)));
  LOSS_CUDA(launch_gather(c.rows, false, c.s));
  LOSS_TRY(c.repack(fn));
  if (!c.maps_of_z()) return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
  c.product.columns = static_cast<int32_t>(d.vocab);
  c.product.part = c.in<float2>(at.part), c.product.target_z = c.in<float>(at.target_z);
  LOSS_CUDA(launch_product<kStats>(c.product, c.s));
  c.rows.part = c.product.part, c.rows.target_z = c.product.target_z;
  c.rows.column_tiles = static_cast<int32_t>(at.column_tiles);
  c.rows.losses = losses, c.rows.lse_out = lse, c.rows.total = total;
  LOSS_CUDA(launch(&k_loss_finish, std::max<int64_t>(1, over(d.tokens, kFinishRows)), kFinishThreads, 0, true, c.s,
                   static_cast<const RowsArgs>(c.rows)));
  return ZERO_OK;
}

extern "C" zero_status zero_linear_cross_entropy_backward(const zero_linear_ce_desc* desc, const void* x,
                                                          const void* w, const void* targets, const float* lse,
                                                          const int32_t* rows, const float* d_loss, int32_t reduction,
                                                          void* dx, void* dw, zero_dtype dw_dtype, void* workspace,
                                                          int64_t workspace_bytes, void* stream) {
  const char* fn = "zero_linear_cross_entropy_backward";
  clear_error();
  NvtxRange range(fn);
  LOSS_TRY(check_desc(fn, desc));
  const zero_linear_ce_desc& d = *desc;
  const bool any = d.tokens > 0;
  if (reduction != ZERO_LOSS_NONE && reduction != ZERO_LOSS_SUM && reduction != ZERO_LOSS_MEAN)
    return fail(ZERO_ERR_INVALID, "%s: unknown reduction", fn);
  if (!known_type(dw_dtype) || (dw_dtype != d.dtype && dw_dtype != ZERO_FP32))
    return fail(ZERO_ERR_INVALID, "%s: dw_dtype must be dtype or ZERO_FP32", fn);
  LOSS_TRY(check_ptr(fn, "x", x, 2, any));
  LOSS_TRY(check_ptr(fn, "w", w, 2, true));
  LOSS_TRY(check_ptr(fn, "targets", targets, d.id_bytes, any));
  LOSS_TRY(check_ptr(fn, "lse", lse, 4, any));
  LOSS_TRY(check_ptr(fn, "rows", rows, 4, true));
  LOSS_TRY(check_ptr(fn, "d_loss", d_loss, 4, any || reduction != ZERO_LOSS_NONE));
  LOSS_TRY(check_ptr(fn, "dx", dx, 2, false));
  LOSS_TRY(check_ptr(fn, "dw", dw, type_bytes(dw_dtype), false));
  LOSS_TRY(check_ptr(fn, "workspace", workspace, 256, true));
  if (!any) dx = nullptr;
  if (!dx && !dw) return ZERO_OK;
  const Layout at(d, wants_repack(d, w), true, true);
  if (workspace_bytes < at.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes,
                at.bytes);
  LOSS_TRY(check_overlaps(fn,
                          {Extent::block("dx", dx, d.tokens * d.hidden * 2),
                           Extent::block("dw", dw, d.vocab * d.hidden * type_bytes(dw_dtype)),
                           Extent::block("workspace", workspace, at.bytes)},
                          {by_rows("x", x, d.tokens, d.x_stride, d.hidden), by_rows("w", w, d.vocab, d.w_stride, d.hidden),
                           Extent::block("targets", targets, d.tokens * d.id_bytes),
                           Extent::block("lse", lse, d.tokens * 4), Extent::block("rows", rows, (d.tokens + 1) * 4),
                           Extent::block("d_loss", d_loss, reduction == ZERO_LOSS_NONE ? d.tokens * 4 : 4)}));
  int32_t* err = nullptr;
  LOSS_TRY(ready(fn, &err));
  Call c(d, at, workspace, stream, w);
  LOSS_TRY(c.begin(fn, x, targets, const_cast<int32_t*>(rows), err));
  c.rows.lse = lse, c.rows.d = d_loss, c.rows.reduction = reduction, c.rows.scale = d.scale;
  c.rows.scales = c.in<Scales>(at.scales), c.rows.lse2 = c.in<float>(at.lse2), c.rows.row_mul = c.in<float>(at.row_mul);
  c.rows.dx = dx;
  c.rows.vec = c.rows.vec && aligned_to(dx, 16);
  LOSS_CUDA(launch(&k_loss_scales, 1, kScanThreads, 0, false, c.s, static_cast<const RowsArgs>(c.rows)));
  LOSS_CUDA(launch_gather(c.rows, true, c.s));
  LOSS_TRY(c.repack(fn));
  if (!c.maps_of_z()) return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
  ProductArgs z = c.product;
  z.lse2 = c.rows.lse2, z.row_mul = c.rows.row_mul, z.dz = c.in<void>(at.dz), z.dz_stride = at.columns;
  for (int64_t first = 0; first < d.vocab; first += at.columns) {
    const int64_t columns = std::min(at.columns, d.vocab - first);
    z.first = static_cast<int32_t>(first), z.columns = static_cast<int32_t>(columns);
    LOSS_CUDA(launch_product<kProbs>(z, c.s));
    ProductArgs p = z;
    p.scales = c.rows.scales;
    if (dx) {
      p.out = dx, p.out_type = d.dtype, p.out_align = align_of(dx, d.hidden * 2);
      p.sums = c.in<float>(at.sums), p.sums_stride = at.sums_stride, p.add = first > 0;
      if (!matrix_map(&p.a, z.dz, c.bf16, columns, at.rows_cap, at.columns, kHalfRows) ||
          !matrix_map(&p.b, c.w, c.bf16, d.hidden, d.vocab, at.w_stride, kTileK))
        return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
      LOSS_CUDA(launch_product<kDx>(p, c.s));
    }
    if (dw) {
      p.out = dw, p.out_type = dw_dtype, p.out_align = align_of(dw, d.hidden * type_bytes(dw_dtype));
      if (!matrix_map(&p.a, z.dz, c.bf16, columns, at.rows_cap, at.columns, kTileK) ||
          !matrix_map(&p.b, c.in<void>(at.xs), c.bf16, d.hidden, at.rows_cap, at.xs_stride, kTileK))
        return fail(ZERO_ERR_CUDA, "%s: the tensor maps could not be made", fn);
      LOSS_CUDA(launch_product<kDw>(p, c.s));
    }
  }
  if (dx) {
    const JoinArgs j = {rows, d.tokens, c.in<float>(at.sums), at.sums_stride, c.rows.scales, dx,
                        static_cast<int32_t>(d.hidden), d.dtype, static_cast<int32_t>(at.columns),
                        static_cast<int32_t>(at.pieces), c.product.pairs};
    LOSS_CUDA(launch(&k_loss_join, kSMs * 8, kGatherThreads, 0, true, c.s, j));
  }
  return ZERO_OK;
}
