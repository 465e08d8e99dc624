// Tokens sorted by expert and brought back with weights, and the gradients.
// Argument checks, kernels, launches.
//
// A token t has `topk` choices; choice k is pair p = t*topk + k with expert
// ids[p].  Choices outside [0, n_experts) are dropped.  The kept pairs, in
// order of (expert, pair), take the rows 0, 1, ..., M-1:
//   offsets[e] = kept pairs of experts below e (offsets[n_experts] = M),
//   rows[p] = p's row or -1, pairs[i] = the pair of row i or -1 past M.
//   dispatch:  xs[rows[p]] = x[t]; the rows past M are zero.
//   combine:   y[t] = sum over k of weights[p] ys[rows[p]], k in order.
//   gradients: dx[t] = sum over k of dxs[rows[p]];
//              dys[rows[p]] = weights[p] dy[t], zero past M;
//              dweights[p] = <dy[t], ys[rows[p]]>, zero for dropped pairs.
// Nothing past row M of ys or dxs is read.
//
// The row kernels are bound by bytes.  They go by token, not by sorted row: a
// token's row is read once and written to its topk places (or gathered from
// them), so each direction moves every byte once, and the sums of a token's
// rows stay in registers in one fixed order.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <inttypes.h>

#include <algorithm>

#include "zero_capi_util.h"
#include "zero_pieces.h"
#include "zero_rows.cuh"

namespace cg = cooperative_groups;

namespace zero {
namespace {

// ---------------------------------------------------------------------------
// The sort: a stable counting sort.  The pairs are cut into one contiguous
// segment a warp; a warp counts its segment's experts in its own shared-memory
// row, the rows are scanned across the warps of all CTAs and the experts, and
// the warp walks its segment again giving out places.  Lanes with the same
// expert find their rank by a warp match, so the order is stable and nothing
// depends on timing.
//
// What bounds it is the walk's latency (32 pairs a step and warp), not bytes.
// Up to kClusterPairs pairs one thread-block cluster does it in one launch,
// its CTAs reading one another's counts through distributed shared memory;
// above, a first launch leaves every CTA's counts in the workspace and up to
// kTableCtas CTAs share the walk.  Cluster and table, us, 64 / 512 experts:
// 32768 pairs 9.9 / 13.5 and 10.9 / 13.7; 49152 pairs 12.1 / 15.6 and 10.1 /
// 13.7; 131072 pairs 22.2 / 28.0 and 13.5 / 16.6.

constexpr int kClusterCtas = 8;        // CTAs of the largest cluster (portable size)
constexpr int64_t kClusterPairs = 32768;
constexpr int kTableCtas = 128;
constexpr int kTableEntries = 65536;   // every CTA reads the whole table
constexpr int kSortWarpsMost = 32;
constexpr int kIdsAhead = 8;
constexpr int kMaxExperts = 4096;
constexpr int kSortSmemMost = 200 * 1024;

struct SortArgs {
  const void* ids;
  int64_t n;           // pairs
  int32_t id_bytes, n_experts;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pairs;
  int32_t* table;      // [CTAs][n_experts]: counts of each CTA's pairs, or null: a cluster
};

__device__ __forceinline__ int load_id(const SortArgs& a, int64_t p) {
  if (a.id_bytes == 4) {
    const int v = static_cast<const int*>(a.ids)[p];
    return v >= 0 && v < a.n_experts ? v : -1;
  }
  const long long v = static_cast<const long long*>(a.ids)[p];
  return v >= 0 && v < a.n_experts ? static_cast<int>(v) : -1;
}

// A warp's pairs among `ctas` CTAs of as many warps: whole groups of 32 but
// for the last warp.
struct Segment {
  int64_t lo, hi;
  __device__ __forceinline__ Segment(int64_t n, int cta, int ctas) {
    const int warps = blockDim.x >> 5;
    const int64_t all = static_cast<int64_t>(ctas) * warps;
    const int64_t size = (((n + all - 1) / all) + 31) / 32 * 32;
    lo = min(n, (static_cast<int64_t>(cta) * warps + (threadIdx.x >> 5)) * size);
    hi = min(n, lo + size);
  }
  // step(expert, pair) for each lane's pairs (expert -1: none or dropped), the
  // ids loaded kIdsAhead groups at a time: the steps depend on one another,
  // their loads need not.
  template <class Step>
  __device__ __forceinline__ void walk(const SortArgs& a, Step step) const {
    const int lane = threadIdx.x & 31;
    for (int64_t p = lo; p < hi; p += 32 * kIdsAhead) {
      int e[kIdsAhead];
#pragma unroll
      for (int i = 0; i < kIdsAhead; ++i) e[i] = p + 32 * i + lane < hi ? load_id(a, p + 32 * i + lane) : -1;
#pragma unroll
      for (int i = 0; i < kIdsAhead; ++i)
        if (p + 32 * i < hi) step(e[i], p + 32 * i + lane);
    }
  }
};

// Every CTA's counts for the walk of many CTAs.
__global__ void __launch_bounds__(32 * kSortWarpsMost) k_expert_count(const SortArgs a) {
  extern __shared__ int smem[];
  let_next_start();
  for (int e = threadIdx.x; e < a.n_experts; e += blockDim.x) smem[e] = 0;
  __syncthreads();
  Segment(a.n, blockIdx.x, gridDim.x).walk(a, [&](int e, int64_t) {
    if (e >= 0) atomicAdd(smem + e, 1);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < a.n_experts; e += blockDim.x)
    a.table[static_cast<int64_t>(blockIdx.x) * a.n_experts + e] = smem[e];
}

template <bool TABLE>
__global__ void __launch_bounds__(32 * kSortWarpsMost) k_expert_sort(const SortArgs a) {
  extern __shared__ int smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int E = a.n_experts;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
  int* count = smem;               // [warps][E]
  int* total = smem + warps * E;   // [E]: this CTA's pairs of each expert
  int* start = total + E;          // [E]: first row of each expert for this CTA
  int* scan = start + E;           // [warps]
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const Segment seg(a.n, me, ctas);
  int* mine = count + warp * E;
  seg.walk(a, [&](int e, int64_t) {
    if (e >= 0) atomicAdd(mine + e, 1);  // only counted here: no order
  });
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int s = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = s;
      s += c;
    }
    total[e] = s;
  }
  if constexpr (TABLE)
    wait_for_previous();
  else
    cluster.sync();
  // the pairs of all CTAs below this one, and of all CTAs, expert by expert;
  // then an exclusive scan of the latter over the experts
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int below = 0, sum = 0;
    if (e < E) {
      if constexpr (TABLE) {
        for (int c0 = 0; c0 < ctas; c0 += 8) {
          int v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = c0 + i < ctas ? __ldcg(a.table + static_cast<int64_t>(c0 + i) * E + e) : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (c0 + i < me) below += v[i];
            sum += v[i];
          }
        }
      } else {
        for (int c = 0; c < ctas; ++c) {
          const int v = cluster.map_shared_rank(total, c)[e];
          if (c < me) below += v;
          sum += v;
        }
      }
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int before = carry, whole = carry;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += scan[w];
      whole += scan[w];
    }
    if (e < E) {
      const int first = before + inc - sum;
      start[e] = first + below;
      if (me == 0) a.offsets[e] = first;
    }
    carry = whole;
    __syncthreads();
  }
  const int M = carry;
  if (me == 0 && threadIdx.x == 0) a.offsets[E] = M;
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] += start[i % E];
  __syncthreads();
  seg.walk(a, [&](int e, int64_t p) {
    const unsigned same = __match_any_sync(kFull, e);
    int row = -1;
    if (e >= 0) row = mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (p < seg.hi) a.rows[p] = row;
    if (row >= 0) a.pairs[row] = static_cast<int>(p);
  });
  for (int64_t i = M + static_cast<int64_t>(me) * blockDim.x + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(ctas) * blockDim.x)
    a.pairs[i] = -1;
  if constexpr (!TABLE) cluster.sync();  // no CTA leaves while another may still read its totals
}

// How a sort is launched.
struct SortShape {
  int ctas, warps, smem;
  bool table;
  SortShape(int64_t n, int n_experts) {
    const int64_t groups = std::max<int64_t>(1, (n + 31) / 32);
    table = n > kClusterPairs;
    // as many warps a CTA as their counters fit, no more than there are groups
    // of 32 pairs, and CTAs until a warp has four groups
    warps = kSortWarpsMost;
    while (warps > 1 && ((warps + 2) * n_experts + warps) * 4 > kSortSmemMost) warps /= 2;
    while (warps > 1 && warps / 2 >= groups) warps /= 2;
    const int most = table ? std::max(8, std::min(kTableCtas, kTableEntries / n_experts)) : kClusterCtas;
    ctas = 1;
    while (ctas < most && static_cast<int64_t>(ctas) * warps * 4 < groups) ctas *= 2;
    smem = ((warps + 2) * n_experts + warps) * 4;
  }
  int64_t table_bytes(int n_experts) const { return table ? static_cast<int64_t>(ctas) * n_experts * 4 : 0; }
};

// ---------------------------------------------------------------------------
// The rows.  A group of 8 to 256 lanes takes a token, octet by octet
// (16-byte aligned rows), or 16-byte pieces and single columns (other rows).
// The rows of all its choices are in flight together, up to 4 (MORE: 4 at a
// time).  (One after the other, the combination of two of 64 experts'
// rows of 4096 bf16, 16384 tokens, took 85 us; together 75; with two columns'
// parts of each as well the registers cost more than the loads gained, 102.)

// Measured, 32768 rows of 4096 bf16 (two a token), us and share of a plain
// copy's bandwidth: dispatch 69 (0.86), its gradient 70 (0.85), combine 75
// (0.79), its gradient 119 (0.83).

constexpr int kRowThreads = 256;
constexpr int kTogether = 4;

// CTAs of an SM that K rows' octets leave registers for.
constexpr int row_ctas(int k, size_t elem, int most) {
  const int held = k * static_cast<int>(elem);  // of a row's eight columns, in pairs of registers
  return held >= 32 ? 2 : held >= 16 ? 3 : held >= 8 ? 4 : most;
}

struct RowArgs {
  const void* in;          // x, ys, dxs or dy
  const void* ys;          // combine's gradient
  const void* weights;     // null: ones
  void* out;               // xs, y, dx or dys
  void* dweights;
  const int32_t* rows;
  const int32_t* total;    // offsets + n_experts
  int64_t tokens, hidden, stride;  // stride: of in's rows (x, dy)
  int32_t topk, weight_type, lanes;
};

// 16 bytes of a row.
template <class T>
struct Piece {
  static constexpr int kCols = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void widen(float (&v)[kCols]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (sizeof(T) == 4)
        v[i] = __uint_as_float(w[i]);
      else
        Elem<T>::unpack(w[i], v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ void narrow(const float (&v)[kCols]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(v[i]);
      else
        w[i] = Elem<T>::pack(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ void store(T* p) const {  // 16-byte aligned
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// 16 bytes that start at any element, as they were loaded: the one or two
// aligned pieces that hold them.  `shifted` puts them together, so that the
// loads of a thread's rows go out before any of them is waited for.
template <class T>
struct Window {
  uint4 a, b;
  __device__ __forceinline__ static int shift(const T* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15); }
  __device__ __forceinline__ void load(const T* p) {
    const int s = shift(p);
    const char* at = reinterpret_cast<const char*>(p) - s;
    a = *reinterpret_cast<const uint4*>(at);
    b = *reinterpret_cast<const uint4*>(at + window_second(s));
  }
  __device__ __forceinline__ Piece<T> shifted(int s) const {
    uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = s & 8 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = s & 4 ? v[i + 1] : v[i];
    Piece<T> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = sizeof(T) == 4 ? v[i] : __funnelshift_r(v[i], v[i + 1], (s & 2) * 8);
    return r;
  }
};

// A row of T's.  A window reaches less than 16 bytes past its columns on
// either side: into the row before or after, but out of the storage from the
// first piece of its first row and the last of its last, which become single
// columns.  Of the rows in expert order the last kept one may end the storage
// and is not known to the combination: there no window passes its row's end.
template <class T>
struct Frame : RowPieces {
  __device__ __forceinline__ Frame(const T* row, int hidden, bool drop_first, bool drop_last)
      : RowPieces(reinterpret_cast<uintptr_t>(row), hidden, static_cast<int>(sizeof(T)), drop_first, drop_last) {}
};
__device__ __forceinline__ uint32_t low_bits(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

// The group's token, and the thread's first column and a round's columns
// where rows are taken octet by octet.
struct Place {
  int64_t token;
  int lane, lanes, first, round;
  __device__ __forceinline__ explicit Place(int lanes_) : lanes(lanes_) {
    token = static_cast<int64_t>(blockIdx.x) * (kRowThreads / lanes) + threadIdx.x / lanes;
    lane = threadIdx.x % lanes;
    first = 8 * lane;
    round = 8 * lanes;
  }
};

// Rows past the last kept pair are zero: the token's own share of them.
template <class T, bool VEC>
__device__ __forceinline__ void clear_past_end(const RowArgs& a, const Place& me, T* out) {
  const int64_t M = __ldg(a.total);
  const int H = static_cast<int>(a.hidden);
  const float z[8] = {};
  for (int k = 0; k < a.topk; ++k) {
    const int64_t i = me.token * a.topk + k;
    if (i < M) continue;
    T* row = out + i * H;
    if constexpr (VEC) {
      for (int c = me.first; c < H; c += me.round) Elem<T>::store8(row + c, z);
    } else {
      const Frame<T> f(row, H, false, false);
      for (int u = me.lane; u < f.pieces; u += me.lanes)
        *reinterpret_cast<uint4*>(row + f.column(u)) = make_uint4(0, 0, 0, 0);
      for (int e = me.lane; e < f.ends; e += me.lanes) row[f.end_column(e)] = Elem<T>::narrow(0.f);
    }
  }
}

// Rows and weights of choices k0 .. k0 + K - 1 of the token whose pairs start
// at p0; -1 past topk.
template <int K>
struct Choices {
  int32_t row[K];
  float weight[K];
  __device__ __forceinline__ Choices(const RowArgs& a, int64_t p0, int k0, bool live) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const bool there = live && k0 + i < a.topk;
      row[i] = there ? __ldg(a.rows + p0 + k0 + i) : -1;
      weight[i] = row[i] >= 0 && a.weights ? load_any(a.weights, p0 + k0 + i, a.weight_type) : 1.f;
    }
  }
};

template <class T, int K, bool MORE>
__global__ void __launch_bounds__(kRowThreads, 6) k_dispatch(const RowArgs a) {
  constexpr int kParts = K == 1 ? 2 : 1;
  const Place me(a.lanes);
  if (me.token >= a.tokens) return;
  const int H = static_cast<int>(a.hidden);
  const T* x = static_cast<const T*>(a.in) + me.token * a.stride;
  T* xs = static_cast<T*>(a.out);
  const int64_t p0 = me.token * a.topk;
  const Choices<K> ch(a, p0, 0, true);
  for (int c0 = me.first; c0 < H; c0 += kParts * me.round) {
    Octet<T> v[kParts];
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      if (c0 + q * me.round < H) v[q].load(x + c0 + q * me.round);
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const int c = c0 + q * me.round;
      if (c >= H) continue;
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (ch.row[i] >= 0) v[q].store(xs + ch.row[i] * static_cast<int64_t>(H) + c);
      for (int k = K; MORE && k < a.topk; ++k) {
        const int64_t r = __ldg(a.rows + p0 + k);
        if (r >= 0) v[q].store(xs + r * H + c);
      }
    }
  }
  clear_past_end<T, true>(a, me, xs);
}

template <class T, int K, bool MORE>
__global__ void __launch_bounds__(kRowThreads, row_ctas(K, sizeof(T), 6)) k_combine(const RowArgs a) {
  constexpr int kParts = K == 1 ? 2 : 1;
  const Place me(a.lanes);
  if (me.token >= a.tokens) return;
  const int H = static_cast<int>(a.hidden);
  const T* in = static_cast<const T*>(a.in);
  T* y = static_cast<T*>(a.out) + me.token * H;
  const int64_t p0 = me.token * a.topk;
  const Choices<K> first(a, p0, 0, !MORE);
  for (int c0 = me.first; c0 < H; c0 += kParts * me.round) {
    float s[kParts][8];
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int n = 0; n < 8; ++n) s[q][n] = 0.f;
    auto add = [&](const Choices<K>& ch) {
      Octet<T> v[kParts][K];
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (ch.row[i] >= 0 && c0 + q * me.round < H)
            v[q][i].load(in + ch.row[i] * static_cast<int64_t>(H) + c0 + q * me.round);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (ch.row[i] >= 0 && c0 + q * me.round < H) {
            float f[8];
            v[q][i].widen(f);
#pragma unroll
            for (int n = 0; n < 8; ++n) s[q][n] = fmaf(ch.weight[i], f[n], s[q][n]);
          }
    };
    if constexpr (MORE) {
#pragma unroll 1
      for (int k0 = 0; k0 < a.topk; k0 += K) add(Choices<K>(a, p0, k0, true));
    } else {
      add(first);
    }
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      if (c0 + q * me.round < H) Elem<T>::store8(y + c0 + q * me.round, s[q]);
  }
}

// Sums of the choices' dots over the group's lanes, to dweights; every thread
// of the CTA is here.
template <int K>
__device__ __forceinline__ void store_dots(const RowArgs& a, const Place& me, bool live, int64_t p0, int k0,
                                           float (&dot)[K], float (&part)[K][kRowThreads / 32]) {
#pragma unroll
  for (int i = 0; i < K; ++i)
    for (int o = min(me.lanes, 32) >> 1; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(kFull, dot[i], o);
  if (me.lanes > 32) {
    // the next choices' sums go to the other half
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) part[i][warp] = dot[i];
    }
    __syncthreads();
    const int warps = me.lanes >> 5, w0 = warp / warps * warps;
    if (me.lane < K) {
      dot[0] = 0.f;
      for (int w = 0; w < warps; ++w) dot[0] += part[me.lane][w0 + w];
    }
  } else {
#pragma unroll
    for (int i = 1; i < K; ++i)
      if (me.lane == i) dot[0] = dot[i];
  }
  if (live && me.lane < K && k0 + me.lane < a.topk)
    store_any(a.dweights, p0 + k0 + me.lane, a.weight_type, dot[0]);
}

template <class T, int K, bool MORE>
__global__ void __launch_bounds__(kRowThreads, row_ctas(K, sizeof(T), 5)) k_combine_backward(const RowArgs a) {
  __shared__ float part[2][K][kRowThreads / 32];
  const Place me(a.lanes);
  const bool live = me.token < a.tokens;  // every thread meets the barriers below
  const int H = static_cast<int>(a.hidden);
  const T* dy = static_cast<const T*>(a.in) + (live ? me.token : 0) * a.stride;
  const T* ys = static_cast<const T*>(a.ys);
  T* dys = static_cast<T*>(a.out);
  const int64_t p0 = (live ? me.token : 0) * a.topk;
  int flip = 0;
  for (int k0 = 0; k0 == 0 || (MORE && k0 < a.topk); k0 += K, flip ^= 1) {
    const Choices<K> ch(a, p0, k0, live);
    float dot[K] = {};
    if (live) {
      for (int c = me.first; c < H; c += me.round) {
        Octet<T> g, v[K];
        g.load(dy + c);
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (ch.row[i] >= 0) v[i].load(ys + ch.row[i] * static_cast<int64_t>(H) + c);
        float d[8];
        g.widen(d);
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (ch.row[i] >= 0) {
            float f[8];
            v[i].widen(f);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              dot[i] = fmaf(d[n], f[n], dot[i]);
              f[n] = d[n] * ch.weight[i];
            }
            Elem<T>::store8(dys + ch.row[i] * static_cast<int64_t>(H) + c, f);
          }
      }
    }
    if (a.dweights) store_dots<K>(a, me, live, p0, k0, dot, part[flip]);
  }
  if (live) clear_past_end<T, true>(a, me, dys);
}

// The same for rows that start anywhere or end inside 16 bytes, by the pieces
// of the rows that are written.
//
// Measured, 16384 tokens, 2 of 64, 4097 bf16, us and share of a plain copy's
// bandwidth; in brackets with eight single columns a thread: dispatch 71
// (0.83) [139], combine 97 (0.61) [119], its gradient 152 (0.65) [388].
// 30000 tokens, 4 of 16, 1001 fp32: dispatch 97 (0.92) [119], the combination's
// gradient 269 (0.58) [351].

template <class T>
__global__ void __launch_bounds__(kRowThreads, 8) k_dispatch_any(const RowArgs a) {
  const Place me(a.lanes);
  if (me.token >= a.tokens) return;
  const int H = static_cast<int>(a.hidden);
  const T* x = static_cast<const T*>(a.in) + me.token * a.stride;
  const bool inner = me.token == 0 || me.token == a.tokens - 1;
  T* xs = static_cast<T*>(a.out);
  const int64_t p0 = me.token * a.topk;
  for (int k = 0; k < a.topk; ++k) {
    const int64_t r = __ldg(a.rows + p0 + k);
    if (r < 0) continue;
    T* row = xs + r * H;
    const Frame<T> f(row, H, inner, inner);
    const int shift = Window<T>::shift(x + f.head);
    T end;
    if (me.lane < f.ends) end = x[f.end_column(me.lane)];
    for (int u = me.lane; u < f.pieces; u += me.lanes) {
      Window<T> v;
      v.load(x + f.column(u));
      v.shifted(shift).store(row + f.column(u));
    }
    if (me.lane < f.ends) row[f.end_column(me.lane)] = end;
    for (int e = me.lane + me.lanes; e < f.ends; e += me.lanes) row[f.end_column(e)] = x[f.end_column(e)];
  }
  clear_past_end<T, false>(a, me, xs);
}

// A thread's single column is loaded before the pieces are waited for (107 us
// at the first size with the loads after them).
template <class T, int K>
__global__ void __launch_bounds__(kRowThreads, K == 1 ? 6 : 5) k_combine_any(const RowArgs a) {
  constexpr int P = Piece<T>::kCols;
  const Place me(a.lanes);
  if (me.token >= a.tokens) return;
  const int H = static_cast<int>(a.hidden);
  const T* in = static_cast<const T*>(a.in);
  T* y = static_cast<T*>(a.out) + me.token * H;
  const Choices<K> ch(a, me.token * a.topk, 0, true);
  const uint32_t row_bytes = static_cast<uint32_t>(H * sizeof(T));
  const uint32_t y_end = low_bits(y) + row_bytes, in_end = low_bits(in) + row_bytes;
  bool first = false, passes = false;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    first |= ch.row[i] == 0;
    passes |= ch.row[i] >= 0 && window_passes(in_end + ch.row[i] * row_bytes, y_end);
  }
  const Frame<T> f(y, H, first, passes);
  T end[K];
  if (me.lane < f.ends)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (ch.row[i] >= 0) end[i] = in[ch.row[i] * static_cast<int64_t>(H) + f.end_column(me.lane)];
  for (int u = me.lane; u < f.pieces; u += me.lanes) {
    const T* from = in + f.column(u);
    float s[P] = {};
    Window<T> v[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (ch.row[i] >= 0) v[i].load(from + ch.row[i] * static_cast<int64_t>(H));
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (ch.row[i] >= 0) {
        float w[P];
        v[i].shifted(Window<T>::shift(from + ch.row[i] * static_cast<int64_t>(H))).widen(w);
#pragma unroll
        for (int n = 0; n < P; ++n) s[n] = fmaf(ch.weight[i], w[n], s[n]);
      }
    Piece<T> out;
    out.narrow(s);
    out.store(y + f.column(u));
  }
  for (int e = me.lane; e < f.ends; e += me.lanes) {
    const int c = f.end_column(e);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (ch.row[i] >= 0)
        s = fmaf(ch.weight[i], Elem<T>::widen(e == me.lane ? end[i] : in[ch.row[i] * static_cast<int64_t>(H) + c]), s);
    y[c] = Elem<T>::narrow(s);
  }
}

// The combination by single columns, eight a thread, `lanes` apart: fp32 rows,
// where a column is a full-rate access and the shift only adds work (30000
// tokens, 4 of 16, 1001 fp32 115 us; by pieces 146), and more than two choices,
// whose windows and sums leave few threads an SM (4 of 16, 1001 bf16 117, by
// pieces 120; 8 of 64, 8000 tokens of 2047 bf16 101, by pieces 148).
template <class T, int K, bool MORE>
__global__ void __launch_bounds__(kRowThreads, K == 4 ? 3 : 4) k_combine_columns(const RowArgs a) {
  const Place me(a.lanes);
  if (me.token >= a.tokens) return;
  const int H = static_cast<int>(a.hidden);
  const T* in = static_cast<const T*>(a.in);
  T* y = static_cast<T*>(a.out) + me.token * H;
  const int64_t p0 = me.token * a.topk;
  const Choices<K> first(a, p0, 0, !MORE);
  for (int c0 = me.lane; c0 < H; c0 += me.round) {
    float s[8] = {};
    auto add = [&](const Choices<K>& ch) {
      T v[K][8];
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (ch.row[i] >= 0) {
          const T* row = in + ch.row[i] * static_cast<int64_t>(H);
#pragma unroll
          for (int n = 0; n < 8; ++n)
            if (c0 + n * me.lanes < H) v[i][n] = row[c0 + n * me.lanes];
        }
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (ch.row[i] >= 0)
#pragma unroll
          for (int n = 0; n < 8; ++n) s[n] = fmaf(ch.weight[i], Elem<T>::widen(v[i][n]), s[n]);
    };
    if constexpr (MORE) {
#pragma unroll 1
      for (int k0 = 0; k0 < a.topk; k0 += K) add(Choices<K>(a, p0, k0, true));
    } else {
      add(first);
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (c0 + n * me.lanes < H) y[c0 + n * me.lanes] = Elem<T>::narrow(s[n]);
  }
}

template <class T, int K, bool MORE>
__global__ void __launch_bounds__(kRowThreads) k_combine_backward_any(const RowArgs a) {
  // a lane has eight columns: two fp32 windows, both in flight
  constexpr int P = Piece<T>::kCols, kParts = sizeof(T) == 4 ? 2 : 1;
  __shared__ float part[2][K][kRowThreads / 32];
  const Place me(a.lanes);
  const bool live = me.token < a.tokens;  // every thread meets the barriers of store_dots
  const int H = static_cast<int>(a.hidden);
  const T* dy = static_cast<const T*>(a.in) + (live ? me.token : 0) * a.stride;
  const T* ys = static_cast<const T*>(a.ys);
  T* dys = static_cast<T*>(a.out);
  const int64_t p0 = (live ? me.token : 0) * a.topk;
  int flip = 0;
  for (int k0 = 0; k0 == 0 || (MORE && k0 < a.topk); k0 += K, flip ^= 1) {
    const Choices<K> ch(a, p0, k0, live);
    float dot[K] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (ch.row[i] < 0) continue;
      const int64_t at = ch.row[i] * static_cast<int64_t>(H);
      const Frame<T> f(dys + at, H, me.token == 0 || ch.row[i] == 0,
                       me.token == a.tokens - 1 || window_passes(low_bits(ys + at + H), low_bits(dys + at + H)));
      const int g_shift = Window<T>::shift(dy + f.head), v_shift = Window<T>::shift(ys + at + f.head);
      for (int u = me.lane; u < f.pieces; u += kParts * me.lanes) {
        Window<T> g[kParts], v[kParts];
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          if (u + q * me.lanes < f.pieces) {
            const int c = f.column(u + q * me.lanes);
            g[q].load(dy + c);
            v[q].load(ys + at + c);
          }
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          if (u + q * me.lanes < f.pieces) {
            float d[P], w[P];
            g[q].shifted(g_shift).widen(d);
            v[q].shifted(v_shift).widen(w);
#pragma unroll
            for (int n = 0; n < P; ++n) {
              dot[i] = fmaf(d[n], w[n], dot[i]);
              w[n] = d[n] * ch.weight[i];
            }
            Piece<T> out;
            out.narrow(w);
            out.store(dys + at + f.column(u + q * me.lanes));
          }
      }
      for (int e = me.lane; e < f.ends; e += me.lanes) {
        const int c = f.end_column(e);
        const float d = Elem<T>::widen(dy[c]);
        dot[i] = fmaf(d, Elem<T>::widen(ys[at + c]), dot[i]);
        dys[at + c] = Elem<T>::narrow(d * ch.weight[i]);
      }
    }
    if (a.dweights) store_dots<K>(a, me, live, p0, k0, dot, part[flip]);
  }
  if (live) clear_past_end<T, false>(a, me, dys);
}

// ---------------------------------------------------------------------------
// host

enum class RowOp { kDispatch, kCombine, kCombineBackward };

template <class T, bool VEC, int K, bool MORE>
int launch_rows_k(RowOp op, const RowArgs& a, cudaStream_t s) {
  // lanes of a token's group: one octet (eight columns) each for as long a
  // row as the CTA allows, a power of two; the gradient's dots want a lane each
  RowArgs copy = a;
  copy.lanes = 8;
  while (copy.lanes < kRowThreads && static_cast<int64_t>(copy.lanes) * 8 < a.hidden) copy.lanes *= 2;
  const int64_t per_cta = kRowThreads / copy.lanes;
  const int64_t grid = (a.tokens + per_cta - 1) / per_cta;
  void* args[] = {&copy};
  const void* fn;
  constexpr bool kByPieces = sizeof(T) == 2 && K <= 2;
  if constexpr (VEC)
    fn = op == RowOp::kDispatch  ? reinterpret_cast<const void*>(&k_dispatch<T, K, MORE>)
         : op == RowOp::kCombine ? reinterpret_cast<const void*>(&k_combine<T, K, MORE>)
                                 : reinterpret_cast<const void*>(&k_combine_backward<T, K, MORE>);
  else if (op == RowOp::kDispatch)
    fn = reinterpret_cast<const void*>(&k_dispatch_any<T>);
  else if (op == RowOp::kCombineBackward)
    fn = reinterpret_cast<const void*>(&k_combine_backward_any<T, K, MORE>);
  else if constexpr (kByPieces)
    fn = reinterpret_cast<const void*>(&k_combine_any<T, K>);
  else
    fn = reinterpret_cast<const void*>(&k_combine_columns<T, K, MORE>);
  return static_cast<int>(cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kRowThreads), args, 0, s));
}

template <class T, bool VEC>
int launch_rows(RowOp op, const RowArgs& a, cudaStream_t s) {
  return a.topk == 1           ? launch_rows_k<T, VEC, 1, false>(op, a, s)
         : a.topk == 2         ? launch_rows_k<T, VEC, 2, false>(op, a, s)
         : a.topk <= kTogether ? launch_rows_k<T, VEC, kTogether, false>(op, a, s)
                               : launch_rows_k<T, VEC, kTogether, true>(op, a, s);
}

template <class T>
int launch_rows_of(RowOp op, const RowArgs& a, cudaStream_t s) {
  const bool vec = a.hidden % 8 == 0 && a.stride * sizeof(T) % 16 == 0 && aligned_to(a.in, 16) &&
                   aligned_to(a.out, 16) && aligned_to(a.ys, 16);
  return vec ? launch_rows<T, true>(op, a, s) : launch_rows<T, false>(op, a, s);
}

zero_status run_rows(const char* fn, RowOp op, const RowArgs& a, zero_dtype dtype, void* stream) {
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int e = dtype == ZERO_FP32   ? launch_rows_of<float>(op, a, s)
                : dtype == ZERO_BF16 ? launch_rows_of<__nv_bfloat16>(op, a, s)
                                     : launch_rows_of<__half>(op, a, s);
  if (e)
    return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(static_cast<cudaError_t>(e)));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return ZERO_OK;
}

zero_status check_sizes(const char* fn, int64_t tokens, int32_t topk) {
  if (tokens < 0 || topk < 1) return fail(ZERO_ERR_INVALID, "%s: need tokens >= 0 and topk >= 1", fn);
  if (tokens > INT32_MAX / topk)
    return fail(ZERO_ERR_INVALID, "%s: tokens * topk must stay below 2^31", fn);
  return ZERO_OK;
}

zero_status check_experts(const char* fn, int32_t n_experts) {
  if (n_experts < 1 || n_experts > kMaxExperts)
    return fail(ZERO_ERR_INVALID, "%s: n_experts must lie in [1, %d]", fn, kMaxExperts);
  return ZERO_OK;
}

zero_status check_rows(const char* fn, int64_t tokens, int32_t topk, int64_t hidden, int dtype) {
  const zero_status st = check_sizes(fn, tokens, topk);
  if (st != ZERO_OK) return st;
  if (hidden < 1 || hidden > INT64_C(1) << 30)
    return fail(ZERO_ERR_INVALID, "%s: hidden must lie in [1, 2^30]", fn);
  if (!known_type(dtype)) return fail(ZERO_ERR_INVALID, "%s: unknown dtype", fn);
  return ZERO_OK;
}

zero_status check_ptr(const char* fn, const char* what, const void* p, int bytes, bool needed) {
  if (needed && !p) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, bytes)) return fail(ZERO_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, what);
  return ZERO_OK;
}

zero_status check_weights(const char* fn, zero_dtype dtype, zero_dtype weight_dtype) {
  if (!known_type(weight_dtype) || (weight_dtype != dtype && weight_dtype != ZERO_FP32))
    return fail(ZERO_ERR_INVALID, "%s: weight_dtype must be dtype or ZERO_FP32", fn);
  return ZERO_OK;
}

// [tokens, hidden] by a stride, [tokens, topk], [n_experts + 1].
Extent token_rows(const char* name, const RowArgs& a, int64_t stride, const void* p, int type) {
  return {name, p, a.tokens, stride * type_bytes(type), a.hidden * type_bytes(type)};
}
Extent choices(const char* name, const RowArgs& a, const void* p, int bytes) {
  return Extent::block(name, p, a.tokens * a.topk * bytes);
}
// Rows in expert order: the last kept one, known on the device, may be the
// last that exists, so only the first is looked at.
Extent sorted_rows(const char* name, const RowArgs& a, const void* p, int type) {
  return Extent::block(name, p, a.hidden * type_bytes(type));
}

#define EXPERT_TRY(x)               \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_expert_sort_workspace_bytes(int64_t tokens, int32_t topk, int32_t n_experts,
                                                        int64_t* bytes) {
  const char* fn = "zero_expert_sort_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  EXPERT_TRY(check_sizes(fn, tokens, topk));
  EXPERT_TRY(check_experts(fn, n_experts));
  *bytes = SortShape(tokens * topk, n_experts).table_bytes(n_experts);
  return ZERO_OK;
}

extern "C" zero_status zero_expert_sort(const void* ids, int32_t id_bytes, int64_t tokens, int32_t topk,
                                        int32_t n_experts, int32_t* offsets, int32_t* rows, int32_t* pairs,
                                        void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "zero_expert_sort";
  clear_error();
  NvtxRange range(fn);
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_ERR_INVALID, "%s: id_bytes must be 4 or 8", fn);
  EXPERT_TRY(check_sizes(fn, tokens, topk));
  EXPERT_TRY(check_experts(fn, n_experts));
  const bool any = tokens > 0;
  EXPERT_TRY(check_ptr(fn, "ids", ids, id_bytes, any));
  EXPERT_TRY(check_ptr(fn, "offsets", offsets, 4, true));
  EXPERT_TRY(check_ptr(fn, "rows", rows, 4, any));
  EXPERT_TRY(check_ptr(fn, "pairs", pairs, 4, any));
  const SortShape shape(tokens * topk, n_experts);
  const int64_t need = shape.table_bytes(n_experts);
  if (need > 0) {
    EXPERT_TRY(check_ptr(fn, "workspace", workspace, 4, true));
    if (workspace_bytes < need)
      return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes,
                  need);
  }
  const int64_t n = tokens * topk;
  EXPERT_TRY(check_overlaps(fn,
                            {Extent::block("offsets", offsets, (n_experts + INT64_C(1)) * 4),
                             Extent::block("rows", rows, n * 4), Extent::block("pairs", pairs, n * 4),
                             Extent::block("workspace", need ? workspace : nullptr, need)},
                            {Extent::block("ids", ids, n * id_bytes)}));
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  const SortArgs a = {ids,  tokens * topk, id_bytes, n_experts,
                      offsets, rows, pairs, shape.table ? static_cast<int32_t*>(workspace) : nullptr};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(shape.ctas);
  cfg.blockDim = dim3(32 * shape.warps);
  cfg.dynamicSmemBytes = shape.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  const void* sort = shape.table ? reinterpret_cast<const void*>(&k_expert_sort<true>)
                                 : reinterpret_cast<const void*>(&k_expert_sort<false>);
  static KernelFacts facts[2];
  e = facts[shape.table].allow(sort, shape.smem, kSortSmemMost);
  if (e == cudaSuccess && shape.table) {
    k_expert_count<<<cfg.gridDim, cfg.blockDim, n_experts * 4, s>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
    // the walk counts its own warps while the counts of the others arrive
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = shape.ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  }
  if (e == cudaSuccess)
    e = shape.table ? cudaLaunchKernelEx(&cfg, k_expert_sort<true>, a)
                    : cudaLaunchKernelEx(&cfg, k_expert_sort<false>, a);
  if (e != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return ZERO_OK;
}

extern "C" zero_status zero_expert_dispatch(const void* x, int64_t x_stride, zero_dtype dtype, int64_t tokens,
                                            int32_t topk, int64_t hidden, const int32_t* offsets,
                                            int32_t n_experts, const int32_t* rows, void* xs, void* stream) {
  const char* fn = "zero_expert_dispatch";
  clear_error();
  NvtxRange range(fn);
  EXPERT_TRY(check_rows(fn, tokens, topk, hidden, dtype));
  EXPERT_TRY(check_experts(fn, n_experts));
  const bool any = tokens > 0;
  EXPERT_TRY(check_ptr(fn, "x", x, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "xs", xs, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "offsets", offsets, 4, any));
  EXPERT_TRY(check_ptr(fn, "rows", rows, 4, any));
  if (any && (x_stride < hidden || x_stride > INT64_C(1) << 40))
    return fail(ZERO_ERR_INVALID, "%s: x_stride must be at least hidden", fn);
  if (!any) return ZERO_OK;
  RowArgs a = {};
  a.in = x, a.out = xs, a.rows = rows, a.total = offsets + n_experts;
  a.tokens = tokens, a.hidden = hidden, a.stride = x_stride, a.topk = topk;
  EXPERT_TRY(check_overlaps(fn, {Extent::block("xs", xs, tokens * topk * hidden * type_bytes(dtype))},
                            {token_rows("x", a, x_stride, x, dtype), choices("rows", a, rows, 4),
                             Extent::block("offsets", offsets, (n_experts + INT64_C(1)) * 4)}));
  return run_rows(fn, RowOp::kDispatch, a, dtype, stream);
}

extern "C" zero_status zero_expert_dispatch_backward(const void* dxs, zero_dtype dtype, int64_t tokens,
                                                     int32_t topk, int64_t hidden, const int32_t* rows,
                                                     void* dx, void* stream) {
  const char* fn = "zero_expert_dispatch_backward";
  clear_error();
  NvtxRange range(fn);
  EXPERT_TRY(check_rows(fn, tokens, topk, hidden, dtype));
  const bool any = tokens > 0;
  EXPERT_TRY(check_ptr(fn, "dxs", dxs, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "dx", dx, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "rows", rows, 4, any));
  if (!any) return ZERO_OK;
  RowArgs a = {};
  a.in = dxs, a.out = dx, a.rows = rows;
  a.tokens = tokens, a.hidden = hidden, a.stride = hidden, a.topk = topk;
  EXPERT_TRY(check_overlaps(fn, {Extent::block("dx", dx, tokens * hidden * type_bytes(dtype))},
                            {sorted_rows("dxs", a, dxs, dtype), choices("rows", a, rows, 4)}));
  return run_rows(fn, RowOp::kCombine, a, dtype, stream);
}

extern "C" zero_status zero_expert_combine(const void* ys, zero_dtype dtype, const void* weights,
                                           zero_dtype weight_dtype, int64_t tokens, int32_t topk,
                                           int64_t hidden, const int32_t* rows, void* y, void* stream) {
  const char* fn = "zero_expert_combine";
  clear_error();
  NvtxRange range(fn);
  EXPERT_TRY(check_rows(fn, tokens, topk, hidden, dtype));
  EXPERT_TRY(check_weights(fn, dtype, weight_dtype));
  const bool any = tokens > 0;
  EXPERT_TRY(check_ptr(fn, "ys", ys, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "weights", weights, type_bytes(weight_dtype), any));
  EXPERT_TRY(check_ptr(fn, "y", y, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "rows", rows, 4, any));
  if (!any) return ZERO_OK;
  RowArgs a = {};
  a.in = ys, a.out = y, a.weights = weights, a.weight_type = weight_dtype, a.rows = rows;
  a.tokens = tokens, a.hidden = hidden, a.stride = hidden, a.topk = topk;
  EXPERT_TRY(check_overlaps(fn, {Extent::block("y", y, tokens * hidden * type_bytes(dtype))},
                            {sorted_rows("ys", a, ys, dtype), choices("rows", a, rows, 4),
                             choices("weights", a, weights, type_bytes(weight_dtype))}));
  return run_rows(fn, RowOp::kCombine, a, dtype, stream);
}

extern "C" zero_status zero_expert_combine_backward(const void* dy, int64_t dy_stride, const void* ys,
                                                    zero_dtype dtype, const void* weights,
                                                    zero_dtype weight_dtype, int64_t tokens, int32_t topk,
                                                    int64_t hidden, const int32_t* offsets,
                                                    int32_t n_experts, const int32_t* rows, void* dys,
                                                    void* dweights, void* stream) {
  const char* fn = "zero_expert_combine_backward";
  clear_error();
  NvtxRange range(fn);
  EXPERT_TRY(check_rows(fn, tokens, topk, hidden, dtype));
  EXPERT_TRY(check_experts(fn, n_experts));
  EXPERT_TRY(check_weights(fn, dtype, weight_dtype));
  const bool any = tokens > 0;
  EXPERT_TRY(check_ptr(fn, "dy", dy, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "ys", ys, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "weights", weights, type_bytes(weight_dtype), any));
  EXPERT_TRY(check_ptr(fn, "dys", dys, type_bytes(dtype), any));
  EXPERT_TRY(check_ptr(fn, "dweights", dweights, type_bytes(weight_dtype), false));
  EXPERT_TRY(check_ptr(fn, "offsets", offsets, 4, any));
  EXPERT_TRY(check_ptr(fn, "rows", rows, 4, any));
  if (any && (dy_stride < hidden || dy_stride > INT64_C(1) << 40))
    return fail(ZERO_ERR_INVALID, "%s: dy_stride must be at least hidden", fn);
  if (!any) return ZERO_OK;
  RowArgs a = {};
  a.in = dy, a.ys = ys, a.weights = weights, a.weight_type = weight_dtype, a.out = dys;
  a.dweights = dweights, a.rows = rows, a.total = offsets + n_experts;
  a.tokens = tokens, a.hidden = hidden, a.stride = dy_stride, a.topk = topk;
  EXPERT_TRY(check_overlaps(fn,
                            {Extent::block("dys", dys, tokens * topk * hidden * type_bytes(dtype)),
                             choices("dweights", a, dweights, type_bytes(weight_dtype))},
                            {token_rows("dy", a, dy_stride, dy, dtype), sorted_rows("ys", a, ys, dtype),
                             choices("weights", a, weights, type_bytes(weight_dtype)), choices("rows", a, rows, 4),
                             Extent::block("offsets", offsets, (n_experts + INT64_C(1)) * 4)}));
  return run_rows(fn, RowOp::kCombineBackward, a, dtype, stream);
}
