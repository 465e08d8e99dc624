// Token embedding and the gradient of its table. Argument checks, kernels,
// launches.
//
//   y[t] = scale * table[ids[t]], 0 for an id outside [0, vocab)
//   dtable[v] (+)= scale * sum of dy[t] over the tokens with ids[t] = v
//
// Both are bound by bytes: every row is read once and written once.
//
// The gradient first puts the tokens in order of their ids, those of one id in
// their own order (k_embed_sort). The sorted tokens are then cut into chunks of
// kChunk, whatever ids they have, so that the work is even however often an id
// occurs (in texts the most frequent are every tenth token); a chunk adds each
// of its runs of equal ids up in binary32 (k_embed_sums) and writes the row,
// or, for a run that goes on in another chunk, a partial row, which k_embed_join
// adds up in order. No atomics but for integer counts: the same call gives the
// same bits. Other CTAs of
// k_embed_sums clear the rows without tokens. (Clearing all rows beforehand: 40 us
// in place of 34 for 32768 tokens, 30522 x 768 fp16; beside the sort it slowed that
// down by more than it took, 43.)
#include <cuda_runtime.h>
#include <inttypes.h>

#include <algorithm>
#include <cmath>

#include "zero_capi_util.h"
#include "zero_rows.cuh"

namespace zero {
namespace {

constexpr int kThreads = 256;
constexpr int kBuckets = 128;       // CTAs of the sort, while an SM's counters hold vocab / kBuckets ids
constexpr int kMinorMost = 1024;
constexpr int kBucketsMost = 4096;  // vocab up to 2^22
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 8;
constexpr int kChunk = 32;  // sorted tokens of a CTA, 16 or 8 where that leaves SMs idle
constexpr int kAhead = 8;  // rows in flight

struct IdsArgs {
  const void* ids;
  int64_t tokens;
  int32_t id_bytes, vocab;
};
// An id as it lies in memory, and what it stands for (-1: outside the table).
template <class I>
__device__ __forceinline__ int row_of(I v, int vocab) {
  return v >= 0 && v < vocab ? static_cast<int>(v) : -1;
}

// Eight values of a row, on a boundary of 16 bytes, binary32 ones of 32: these
// move by 32 bytes, because by 16 a warp's access touches twice the lines for
// half of each.
template <class P>
__device__ __forceinline__ void load_row8(const P* p, Octet<P>& o) {
  if constexpr (sizeof(P) == 4)
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(o.w[0].x), "=r"(o.w[0].y), "=r"(o.w[0].z), "=r"(o.w[0].w), "=r"(o.w[1].x), "=r"(o.w[1].y),
                   "=r"(o.w[1].z), "=r"(o.w[1].w)
                 : "l"(p)
                 : "memory");
  else
    o.load(p);
}
template <class P>
__device__ __forceinline__ void store_row8(P* p, const float (&v)[8]) {
  if constexpr (sizeof(P) == 4)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  else
    Elem<P>::store8(p, v);
}

// ---------------------------------------------------------------------------
// lookup

struct LookupArgs {
  IdsArgs ids;
  const void* table;
  void* y;
  int64_t stride;
  int32_t hidden;
  float scale;
};

// A CTA's rows of threads (x: a token's octets, y: tokens) take TOKENS
// neighbouring tokens each, all their rows in flight together. One token leaves a
// row's loads alone in flight behind that of its id: 24 us for 32768 tokens of
// 768 fp16 and 64 us for 16384 of 4096 bf16 to fp32, with four 12 and 52 (0.77 and
// 0.91 of a plain copy's bandwidth).
template <class I, class T, class Y, int TOKENS>
__global__ void __launch_bounds__(kThreads) k_embed(const LookupArgs a) {
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y) * TOKENS;
  if (t0 >= a.ids.tokens) return;
  const I* ids = static_cast<const I*>(a.ids.ids);
  I raw[TOKENS];
#pragma unroll
  for (int k = 0; k < TOKENS; ++k) raw[k] = ids[min(t0 + k, a.ids.tokens - 1)];
  const T* row[TOKENS];
#pragma unroll
  for (int k = 0; k < TOKENS; ++k) {
    const int id = row_of(raw[k], a.ids.vocab);
    row[k] = id >= 0 ? static_cast<const T*>(a.table) + id * a.stride : nullptr;
  }
  Y* y = static_cast<Y*>(a.y) + t0 * a.hidden;
  for (int c = 8 * threadIdx.x; c < a.hidden; c += 8 * blockDim.x) {
    Octet<T> v[TOKENS];
#pragma unroll
    for (int k = 0; k < TOKENS; ++k)
      if (row[k]) load_row8(row[k] + c, v[k]);
#pragma unroll
    for (int k = 0; k < TOKENS; ++k)
      if (t0 + k < a.ids.tokens) {
        float f[8] = {};
        if (row[k]) {
          v[k].widen(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= a.scale;
        }
        store_row8(y + static_cast<int64_t>(k) * a.hidden + c, f);
      }
  }
}

// Rows that start anywhere: single columns, eight a thread.
template <class I, class T, class Y>
__global__ void __launch_bounds__(kThreads) k_embed_any(const LookupArgs a) {
  const int lanes = blockDim.x, lane = threadIdx.x;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.ids.tokens) return;
  const int id = row_of(static_cast<const I*>(a.ids.ids)[t], a.ids.vocab);
  Y* y = static_cast<Y*>(a.y) + t * a.hidden;
  const T* row = static_cast<const T*>(a.table) + id * a.stride;
  for (int c0 = lane; c0 < a.hidden; c0 += 8 * lanes) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (id >= 0 && c0 + i * lanes < a.hidden) v[i] = row[c0 + i * lanes];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i * lanes < a.hidden)
        y[c0 + i * lanes] = Elem<Y>::narrow(id >= 0 ? Elem<T>::widen(v[i]) * a.scale : 0.f);
  }
}

// ---------------------------------------------------------------------------
// gradient

struct SortArgs {
  IdsArgs ids;
  int32_t bits, minors;  // id = minor << bits | bucket
  int2* order;           // sorted: token and id
  int32_t* starts;       // [buckets * minors + 1]: first place of each id, by (bucket, minor)
};

// One CTA a bucket of ids (id mod the number of CTAs: the frequent ids, which
// have small numbers, fall into different ones). Every CTA looks at all ids:
// counts its own, warp by warp, and those of the buckets before it, and keeps
// its own in a list for each warp; then goes through the lists and gives out
// places, which are in the tokens' order because a warp's tokens are
// consecutive. (A CTA with a full list goes through the ids again.) Nothing
// passes between CTAs, so it is one launch and no order depends on timing; what
// it costs is one read of the ids from L2 for each bucket.
constexpr int kListed = 256;        // of a warp's list
constexpr int kMinorBits = 10;      // of an entry; the rest is the place among the warp's tokens
static_assert(kMinorMost == 1 << kMinorBits, "an entry's parts");

template <class I>
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const SortArgs a) {
  extern __shared__ int count[];  // [kSortWarps][minors], then first places; [minors]: the ids' first places
  __shared__ uint32_t list[kSortWarps][kListed];
  __shared__ int below[kSortWarps], scan[kSortWarps];
  let_next_start();
  const I* ids = static_cast<const I*>(a.ids.ids);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bucket = blockIdx.x, mask = (1 << a.bits) - 1, minors = a.minors;
  const unsigned lower = (1u << lane) - 1;
  int* first = count + kSortWarps * minors;
  for (int i = threadIdx.x; i < kSortWarps * minors; i += kSortThreads) count[i] = 0;
  __syncthreads();
  const int64_t size = ((a.ids.tokens + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t lo = min(a.ids.tokens, warp * size), hi = min(a.ids.tokens, lo + size);
  int* mine = count + warp * minors;
  int before = 0, listed = 0;
  for (int64_t p = lo; p < hi; p += 32 * kSortAhead) {
    I raw[kSortAhead];
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) raw[i] = ids[min(p + 32 * i + lane, hi - 1)];
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      const int id = p + 32 * i + lane < hi ? row_of(raw[i], a.ids.vocab) : -1;
      const int b = id & mask;
      before += id >= 0 && b < bucket;
      const bool own = id >= 0 && b == bucket;
      const unsigned owners = __ballot_sync(kFull, own);
      if (!owners) continue;
      if (own) {
        const int m = id >> a.bits, at = listed + __popc(owners & lower);
        atomicAdd(mine + m, 1);  // only counted here: no order
        if (at < kListed) list[warp][at] = static_cast<uint32_t>(p - lo + 32 * i + lane) << kMinorBits | m;
      }
      listed += __popc(owners);
    }
  }
  before = __reduce_add_sync(kFull, before);
  if (lane == 0) below[warp] = before;
  __syncthreads();
  before = __reduce_add_sync(kFull, below[lane]);
  // places of every warp's tokens of an id, and the ids' totals
  int carry = before;
  for (int m0 = 0; m0 < minors; m0 += kSortThreads) {
    const int m = m0 + threadIdx.x;
    int sum = 0;
    if (m < minors)
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = count[w * minors + m];
        count[w * minors + m] = sum;
        sum += c;
      }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int at = carry + inc - sum;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) at += scan[w];
      carry += scan[w];
    }
    if (m < minors) {
      first[m] = at;
      a.starts[static_cast<int64_t>(bucket) * minors + m] = at;
    }
    __syncthreads();
  }
  if (bucket == static_cast<int>(gridDim.x) - 1 && threadIdx.x == 0)
    a.starts[static_cast<int64_t>(gridDim.x) * minors] = carry;
  // places of 32 of the warp's tokens (m -1: not this bucket's)
  auto place = [&](int64_t token, int m) {
    const unsigned owners = __ballot_sync(kFull, m >= 0);
    if (m >= 0) {
      const unsigned same = __match_any_sync(owners, m);
      const int rank = __popc(same & lower);
      const int at = first[m] + mine[m] + rank;
      __syncwarp(owners);
      if (rank == 0) mine[m] += __popc(same);
      a.order[at] = make_int2(static_cast<int>(token), m << a.bits | bucket);
    }
    __syncwarp();
  };
  if (listed <= kListed && size <= INT64_C(1) << (32 - kMinorBits)) {
    for (int i = lane; i - lane < listed; i += 32) {
      const uint32_t e = i < listed ? list[warp][i] : 0;
      place(lo + (e >> kMinorBits), i < listed ? static_cast<int>(e & (kMinorMost - 1)) : -1);
    }
  } else {
    for (int64_t p = lo; p < hi; p += 32 * kSortAhead) {
      I raw[kSortAhead];
#pragma unroll
      for (int i = 0; i < kSortAhead; ++i) raw[i] = ids[min(p + 32 * i + lane, hi - 1)];
#pragma unroll
      for (int i = 0; i < kSortAhead; ++i) {
        const int id = p + 32 * i + lane < hi ? row_of(raw[i], a.ids.vocab) : -1;
        place(p + 32 * i + lane, id >= 0 && (id & mask) == bucket ? id >> a.bits : -1);
      }
    }
  }
}

struct SumArgs {
  const int2* order;
  const int32_t* starts;
  int32_t total_at;      // starts[total_at]: sorted tokens
  int32_t bits, minors;
  const void* dy;
  int64_t dy_stride, part_stride;
  void* out;
  float* part;           // [chunks][2][part_stride]: of a run from an earlier chunk, of a run that goes on
  int2* tail;            // [chunks]: the id that begins in a chunk and goes on (-1: none), chunks that it goes on in
  int32_t hidden, out_type, add, vocab, chunk;
  int64_t chunks;
  float scale;
};

// What a thread holds of a row: an octet, or eight columns `step` apart.
template <bool VEC>
struct Columns {
  int c0, step, hidden;
  __device__ __forceinline__ bool any() const { return c0 < hidden; }
  __device__ __forceinline__ int at(int i) const { return c0 + (VEC ? i : i * step); }
  __device__ __forceinline__ bool in(int i) const { return VEC || at(i) < hidden; }
  // As it was loaded, so that several rows' loads go out before any is used.
  template <class P>
  struct Raw {
    Octet<P> octet;
    P one[VEC ? 1 : 8];
  };
  template <class P>
  __device__ __forceinline__ void load(const P* row, Raw<P>& r) const {
    if constexpr (VEC) {
      load_row8(row + c0, r.octet);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.one[i] = row[in(i) ? at(i) : 0];
    }
  }
  template <class P>
  __device__ __forceinline__ void widen(const Raw<P>& r, float (&v)[8]) const {
    if constexpr (VEC) {
      r.octet.widen(v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = Elem<P>::widen(r.one[i]);
    }
  }
  template <class P>
  __device__ __forceinline__ void store(P* row, const float (&v)[8]) const {
    if constexpr (VEC) {
      store_row8(row + c0, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in(i)) row[at(i)] = Elem<P>::narrow(v[i]);
    }
  }
  // scale * sum, on top of what is there
  template <class P>
  __device__ __forceinline__ void finish(P* row, const float (&sum)[8], float scale, bool add) const {
    float v[8] = {};
    if (add) {
      Raw<P> r;
      load(row, r);
      widen(r, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(scale, sum[i], v[i]);
    store(row, v);
  }
  __device__ __forceinline__ void clear_any(const SumArgs& a, int id) const {
    const int64_t row = static_cast<int64_t>(id) * a.hidden;
    const float zero[8] = {};
    if (a.out_type == ZERO_FP32)
      store(static_cast<float*>(a.out) + row, zero);
    else  // 0 is 0 in both 16-bit types
      store(static_cast<__half*>(a.out) + row, zero);
  }
  __device__ __forceinline__ void finish_any(const SumArgs& a, int id, const float (&sum)[8]) const {
    const int64_t row = static_cast<int64_t>(id) * a.hidden;
    if (a.out_type == ZERO_FP32)
      finish(static_cast<float*>(a.out) + row, sum, a.scale, a.add);
    else if (a.out_type == ZERO_BF16)
      finish(static_cast<__nv_bfloat16*>(a.out) + row, sum, a.scale, a.add);
    else
      finish(static_cast<__half*>(a.out) + row, sum, a.scale, a.add);
  }
};

// A chunk's sums. The rows are loaded AHEAD at a time, whichever runs they
// belong to; the runs' ends are the same for every thread.
constexpr int kClearRows = 8;  // that a CTA looks at
template <class D, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_sums(const SumArgs a) {
  constexpr int AHEAD = VEC ? kAhead : 4;
  __shared__ int2 item[kChunk + 2];
  let_next_start();
  wait_for_previous();
  const Columns<VEC> cols = {VEC ? static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x) * 8
                                 : static_cast<int>(blockIdx.y * blockDim.x * 8 + threadIdx.x),
                             static_cast<int>(blockDim.x), a.hidden};
  if (blockIdx.x >= a.chunks) {
    const int first = static_cast<int>(blockIdx.x - a.chunks) * kClearRows;
    bool empty[kClearRows];
#pragma unroll
    for (int i = 0; i < kClearRows; ++i) {
      const int id = min(first + i, a.vocab - 1);
      const int64_t at = static_cast<int64_t>(id & ((1 << a.bits) - 1)) * a.minors + (id >> a.bits);
      empty[i] = a.starts[at] == a.starts[at + 1];
    }
#pragma unroll
    for (int i = 0; i < kClearRows; ++i)
      if (empty[i] && first + i < a.vocab && cols.any()) cols.clear_any(a, first + i);
    return;
  }
  const int total = a.starts[a.total_at];
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  if (lo >= total) {
    if (blockIdx.y == 0 && threadIdx.x == 0) a.tail[blockIdx.x] = make_int2(-1, 0);
    return;
  }
  const int n = static_cast<int>(min(static_cast<int64_t>(a.chunk), total - lo));
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const int64_t p = lo + i - 1;
    item[i] = p >= 0 && p < total ? a.order[p] : make_int2(-1, -1);
  }
  __syncthreads();
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    int2 tail = make_int2(-1, 0);
    const int id = item[n].y;
    if (item[n + 1].y == id) {
      const int64_t at = static_cast<int64_t>(id & ((1 << a.bits) - 1)) * a.minors + (id >> a.bits);
      if (a.starts[at] >= lo) tail = make_int2(id, (a.starts[at + 1] - 1) / a.chunk - static_cast<int>(blockIdx.x));
    }
    a.tail[blockIdx.x] = tail;
  }
  if (!cols.any()) return;
  const D* dy = static_cast<const D*>(a.dy);
  float sum[8] = {};
  int run_from = 0;
  for (int i0 = 0; i0 < n; i0 += AHEAD) {
    typename Columns<VEC>::template Raw<D> raw[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) cols.load(dy + item[min(i0 + k, n - 1) + 1].x * a.dy_stride, raw[k]);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k;
      if (i >= n) break;
      float v[8];
      cols.widen(raw[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
      const int id = item[i + 1].y;
      const bool goes_on = item[i + 2].y == id;
      if (goes_on && i + 1 < n) continue;
      const bool from_before = run_from == 0 && item[0].y == id;
      if (from_before || goes_on)
        cols.store(a.part + (blockIdx.x * INT64_C(2) + (from_before ? 0 : 1)) * a.part_stride, sum);
      else
        cols.finish_any(a, id, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.f;
      run_from = i + 1;
    }
  }
}

// Runs over several chunks: the chunk in which one begins adds its parts up,
// kJoinGroups threads a column, each a contiguous share of the chunks.
constexpr int kJoinLanes = 64, kJoinGroups = kThreads / kJoinLanes;
template <bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(const SumArgs a) {
  __shared__ float part[kJoinGroups][8][kJoinLanes];
  wait_for_previous();
  const int64_t chunk = blockIdx.x;
  const int2 tail = a.tail[chunk];
  const int id = tail.x, parts = tail.y;  // parts: chunks after this one
  if (id < 0) return;
  const int lane = threadIdx.x % kJoinLanes, g = threadIdx.x / kJoinLanes;
  const Columns<VEC> cols = {VEC ? static_cast<int>(blockIdx.y * kJoinLanes + lane) * 8
                                 : static_cast<int>(blockIdx.y * kJoinLanes * 8 + lane),
                             kJoinLanes, a.hidden};
  float sum[8] = {};
  if (cols.any()) {
    constexpr int AHEAD = VEC ? 4 : 2;
    const int each = (parts + kJoinGroups - 1) / kJoinGroups, k1 = min(parts, (g + 1) * each);
    typename Columns<VEC>::template Raw<float> raw[AHEAD];
    if (g == 0) {
      cols.load(a.part + (chunk * 2 + 1) * a.part_stride, raw[0]);
      cols.widen(raw[0], sum);
    }
    for (int k = g * each; k < k1; k += AHEAD) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) cols.load(a.part + (chunk + 1 + min(k + q, k1 - 1)) * 2 * a.part_stride, raw[q]);
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        if (k + q >= k1) break;
        float v[8];
        cols.widen(raw[q], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[g][j][lane] = sum[j];
  __syncthreads();
  if (g == 0 && cols.any()) {
    for (int k = 1; k < kJoinGroups; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += part[k][j][lane];
    cols.finish_any(a, id, sum);
  }
}

// ---------------------------------------------------------------------------
// host

template <class... P>
cudaError_t launch(void (*fn)(P...), dim3 grid, dim3 threads, size_t smem, bool early, cudaStream_t s, P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
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

// One token a row of threads while that leaves SMs without a CTA, else four.
template <class I, class T, class Y>
cudaError_t launch_lookup(const LookupArgs& a, bool vec, cudaStream_t s) {
  const int units = (a.hidden + 7) / 8, rounds = (units + kThreads - 1) / kThreads;
  const int lanes = (units + rounds - 1) / rounds, rows = kThreads / lanes;
  const int64_t one = (a.ids.tokens + rows - 1) / rows;
  const bool four = vec && one >= 8 * kSMs;
  const int64_t grid = four ? (a.ids.tokens + 4 * rows - 1) / (4 * rows) : one;
  return launch(four  ? &k_embed<I, T, Y, 4>
                : vec ? &k_embed<I, T, Y, 1>
                      : &k_embed_any<I, T, Y>,
                dim3(static_cast<unsigned>(grid)), dim3(lanes, rows), 0, false, s, a);
}
template <class T, class Y>
cudaError_t launch_lookup(const LookupArgs& a, bool vec, cudaStream_t s) {
  return a.ids.id_bytes == 4 ? launch_lookup<int32_t, T, Y>(a, vec, s) : launch_lookup<long long, T, Y>(a, vec, s);
}

// The workspace of the gradient.
struct Layout {
  int bits, minors, buckets, chunk;
  int64_t chunks, part_stride, order, starts, tail, part, bytes;
  Layout(int64_t tokens, int64_t vocab, int64_t hidden) {
    buckets = kBuckets, bits = 7;
    while ((vocab + buckets - 1) / buckets > kMinorMost) buckets *= 2, ++bits;
    minors = static_cast<int>((vocab + buckets - 1) / buckets);
    const int64_t ctas = (hidden + 8 * kThreads - 1) / (8 * kThreads);  // of a chunk
    chunk = kChunk;
    while (chunk > 8 && (tokens + chunk - 1) / chunk * ctas < 4 * kSMs) chunk /= 2;
    chunks = (tokens + chunk - 1) / chunk;
    part_stride = (hidden + 7) / 8 * 8;
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    order = 0;
    starts = up(tokens * 8);
    tail = starts + up((static_cast<int64_t>(buckets) * minors + 1) * 4);
    part = tail + up(chunks * 8);
    bytes = part + chunks * 2 * part_stride * 4;
  }
  int sort_smem() const { return (kSortWarps + 1) * minors * 4; }
};
constexpr int kSortSmemMost = (kSortWarps + 1) * kMinorMost * 4;

template <class D, bool VEC>
cudaError_t launch_sums(const SumArgs& a, int64_t chunks, cudaStream_t s) {
  const int units = static_cast<int>((a.hidden + 7) / 8);  // threads that a row takes
  // CTAs of as many warps as a row's columns fill, evenly when it takes several
  const int ctas = (units + kThreads - 1) / kThreads;
  const int threads = ((units + ctas - 1) / ctas + 31) / 32 * 32;
  const int64_t clear = a.add ? 0 : (a.vocab + kClearRows - 1) / kClearRows;
  cudaError_t e = launch(&k_embed_sums<D, VEC>, dim3(static_cast<unsigned>(chunks + clear), ctas), threads, 0, true, s, a);
  if (e == cudaSuccess && chunks > 1)
    e = launch(&k_embed_join<VEC>, dim3(static_cast<unsigned>(chunks - 1), (units + kJoinLanes - 1) / kJoinLanes),
               kThreads, 0, true, s, a);
  return e;
}

zero_status check_sizes(const char* fn, int64_t tokens, int64_t vocab, int64_t hidden) {
  if (tokens < 0 || tokens > INT64_C(1) << 28)
    return fail(ZERO_ERR_INVALID, "%s: tokens must lie in [0, 2^28]", fn);
  if (vocab < 1 || vocab > static_cast<int64_t>(kBucketsMost) * kMinorMost)
    return fail(ZERO_ERR_INVALID, "%s: vocab must lie in [1, 2^22]", fn);
  if (hidden < 1 || hidden > INT64_C(1) << 20) return fail(ZERO_ERR_INVALID, "%s: hidden must lie in [1, 2^20]", fn);
  return ZERO_OK;
}

zero_status check_ptr(const char* fn, const char* what, const void* p, int bytes, bool needed) {
  if (needed && !p) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, bytes)) return fail(ZERO_ERR_ALIGN, "%s: %s is not aligned to %d bytes", fn, what, bytes);
  return ZERO_OK;
}

zero_status check_common(const char* fn, int32_t id_bytes, double scale, int64_t stride, int64_t hidden) {
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_ERR_INVALID, "%s: id_bytes must be 4 or 8", fn);
  if (!std::isfinite(scale) || !std::isfinite(static_cast<float>(scale)))
    return fail(ZERO_ERR_INVALID, "%s: scale must be finite", fn);
  if (stride < hidden || stride > INT64_C(1) << 36)
    return fail(ZERO_ERR_INVALID, "%s: strides must be at least hidden", fn);
  return ZERO_OK;
}

// Rows that are taken octet by octet.
bool wide_rows(int64_t hidden, const void* p, int64_t stride, int bytes) {
  return hidden % 8 == 0 && stride % 8 == 0 && aligned_to(p, 8 * bytes);
}

zero_status pending_error(const char* fn) {
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  return ZERO_OK;
}

#define EMBED_TRY(x)                \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_embedding(const void* ids, int32_t id_bytes, int64_t tokens, const void* table,
                                      int64_t table_stride, zero_dtype table_dtype, int64_t vocab, int64_t hidden,
                                      double scale, void* y, zero_dtype y_dtype, void* stream) {
  const char* fn = "zero_embedding";
  clear_error();
  NvtxRange range(fn);
  EMBED_TRY(check_sizes(fn, tokens, vocab, hidden));
  EMBED_TRY(check_common(fn, id_bytes, scale, table_stride, hidden));
  if (!known_type(table_dtype)) return fail(ZERO_ERR_INVALID, "%s: unknown table_dtype", fn);
  if (y_dtype != table_dtype && y_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: y_dtype must be table_dtype or ZERO_FP32", fn);
  const bool any = tokens > 0;
  EMBED_TRY(check_ptr(fn, "ids", ids, id_bytes, any));
  EMBED_TRY(check_ptr(fn, "table", table, type_bytes(table_dtype), any));
  EMBED_TRY(check_ptr(fn, "y", y, type_bytes(y_dtype), any));
  if (!any) return ZERO_OK;
  const int e = type_bytes(table_dtype);
  EMBED_TRY(check_overlaps(fn, {Extent::block("y", y, tokens * hidden * type_bytes(y_dtype))},
                           {{"table", table, vocab, table_stride * e, hidden * e},
                            Extent::block("ids", ids, tokens * id_bytes)}));
  EMBED_TRY(pending_error(fn));
  LookupArgs a = {{ids, tokens, id_bytes, static_cast<int32_t>(vocab)}, table, y, table_stride,
                  static_cast<int32_t>(hidden), static_cast<float>(scale)};
  const bool vec = wide_rows(hidden, table, table_stride, e) && wide_rows(hidden, y, hidden, type_bytes(y_dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = y_dtype == ZERO_FP32;
  const cudaError_t r = table_dtype == ZERO_FP32   ? launch_lookup<float, float>(a, vec, s)
                        : table_dtype == ZERO_BF16 ? (wide ? launch_lookup<__nv_bfloat16, float>(a, vec, s)
                                                           : launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, s))
                        : wide                     ? launch_lookup<__half, float>(a, vec, s)
                                                   : launch_lookup<__half, __half>(a, vec, s);
  if (r != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(r));
  return ZERO_OK;
}

extern "C" zero_status zero_embedding_workspace_bytes(int64_t tokens, int64_t vocab, int64_t hidden, int64_t* bytes) {
  const char* fn = "zero_embedding_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  EMBED_TRY(check_sizes(fn, tokens, vocab, hidden));
  *bytes = Layout(tokens, vocab, hidden).bytes;
  return ZERO_OK;
}

extern "C" zero_status zero_embedding_backward(const void* dy, int64_t dy_stride, zero_dtype dy_dtype,
                                               const void* ids, int32_t id_bytes, int64_t tokens, int64_t vocab,
                                               int64_t hidden, double scale, int32_t accumulate, void* dtable,
                                               zero_dtype dtable_dtype, void* workspace, int64_t workspace_bytes,
                                               void* stream) {
  const char* fn = "zero_embedding_backward";
  clear_error();
  NvtxRange range(fn);
  EMBED_TRY(check_sizes(fn, tokens, vocab, hidden));
  EMBED_TRY(check_common(fn, id_bytes, scale, dy_stride, hidden));
  if (!known_type(dy_dtype) || !known_type(dtable_dtype)) return fail(ZERO_ERR_INVALID, "%s: unknown dtype", fn);
  if (dy_dtype != dtable_dtype && dy_dtype != ZERO_FP32 && dtable_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: dy and dtable must have one type, or one of them ZERO_FP32", fn);
  const bool any = tokens > 0;
  const Layout at(tokens, vocab, hidden);
  EMBED_TRY(check_ptr(fn, "dy", dy, type_bytes(dy_dtype), any));
  EMBED_TRY(check_ptr(fn, "ids", ids, id_bytes, any));
  EMBED_TRY(check_ptr(fn, "dtable", dtable, type_bytes(dtable_dtype), true));
  EMBED_TRY(check_ptr(fn, "workspace", workspace, 256, any));
  if (any && workspace_bytes < at.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes,
                at.bytes);
  const int e = type_bytes(dy_dtype);
  const int64_t out_bytes = vocab * hidden * type_bytes(dtable_dtype);
  EMBED_TRY(check_overlaps(
      fn, {Extent::block("dtable", dtable, out_bytes), Extent::block("workspace", any ? workspace : nullptr, at.bytes)},
      {{"dy", dy, tokens, dy_stride * e, hidden * e}, Extent::block("ids", ids, tokens * id_bytes)}));
  if (!any && accumulate) return ZERO_OK;
  EMBED_TRY(pending_error(fn));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t r = cudaSuccess;
  if (!any) {
    r = cudaMemsetAsync(dtable, 0, out_bytes, s);
    if (r != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: clearing failed: %s", fn, cudaGetErrorString(r));
    return ZERO_OK;
  }
  char* ws = static_cast<char*>(workspace);
  const SortArgs sort = {{ids, tokens, id_bytes, static_cast<int32_t>(vocab)}, at.bits, at.minors,
                         reinterpret_cast<int2*>(ws + at.order), reinterpret_cast<int32_t*>(ws + at.starts)};
  static KernelFacts facts[2];
  auto* sort_fn = id_bytes == 4 ? &k_embed_sort<int32_t> : &k_embed_sort<long long>;
  r = facts[id_bytes == 4].allow(reinterpret_cast<const void*>(sort_fn), kSortSmemMost, kSortSmemMost);
  if (r == cudaSuccess) r = launch(sort_fn, dim3(at.buckets), kSortThreads, at.sort_smem(), false, s, sort);
  SumArgs a = {};
  a.order = sort.order, a.starts = sort.starts, a.total_at = at.buckets * at.minors;
  a.bits = at.bits, a.minors = at.minors, a.dy = dy, a.dy_stride = dy_stride, a.part_stride = at.part_stride;
  a.out = dtable, a.part = reinterpret_cast<float*>(ws + at.part), a.hidden = static_cast<int32_t>(hidden);
  a.out_type = dtable_dtype, a.add = accumulate != 0, a.vocab = static_cast<int32_t>(vocab);
  a.scale = static_cast<float>(scale), a.tail = reinterpret_cast<int2*>(ws + at.tail), a.chunk = at.chunk, a.chunks = at.chunks;
  const bool vec = wide_rows(hidden, dy, dy_stride, e) && wide_rows(hidden, dtable, hidden, type_bytes(dtable_dtype));
  if (r == cudaSuccess)
    r = dy_dtype == ZERO_FP32   ? (vec ? launch_sums<float, true>(a, at.chunks, s)
                                       : launch_sums<float, false>(a, at.chunks, s))
        : dy_dtype == ZERO_BF16 ? (vec ? launch_sums<__nv_bfloat16, true>(a, at.chunks, s)
                                       : launch_sums<__nv_bfloat16, false>(a, at.chunks, s))
        : vec                   ? launch_sums<__half, true>(a, at.chunks, s)
                                : launch_sums<__half, false>(a, at.chunks, s);
  if (r != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(r));
  return ZERO_OK;
}
