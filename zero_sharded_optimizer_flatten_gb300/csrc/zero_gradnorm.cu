// Norm of the gradients of many tensors as if they were one vector, and the
// clipping that goes with it: argument checks, job tables, kernels, launches.
//
// Mathematics.  norm = sqrt(sum g^2) (or max |g|) over every element of every
// tensor, c = min(1, max_norm / (norm + 1e-6)), dst = c * src, the product in
// binary32 and rounded once to dst's type.
//
// What bounds it: bytes.  The norm reads every gradient once, the clipping
// reads them again and writes them; nothing can be written before the last
// element is read.
//
// Work split.  A tensor is cut into tiles of 8192 elements, a CTA takes a
// contiguous run of tiles (of any tensors) and leaves one partial,
// so the partials are few (at most kGrid a launch) and every CTA of the
// clipping adds them up itself, in the same fixed order: no kernel between
// the two passes, no atomics, the same norm in every run.  A thread has
// 128 bytes of loads in flight.  The clipping walks the tiles from
// the last to the first, so what the norm read last is still in L2, and it is
// launched early (its CTAs wait for the norm's on the device).
#include <cuda_runtime.h>
#include <inttypes.h>
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "zero_capi_util.h"
#include "zero_rows.cuh"

namespace zero {
namespace {

constexpr int kNormThreads = 128;
constexpr int kNormTile = 8192;                        // elements a CTA takes at once
constexpr int kTileOctets = kNormTile / 8;             // 1024
constexpr int kAhead = kTileOctets / kNormThreads;     // octets of a thread: 8
// Bytes of a thread's loads in flight.  64, with more CTAs an SM: the norm of
// 212M fp32 values 141 us, bf16 82; 128: 127 and 71.
constexpr int kBytesAhead = 128;
constexpr int kNormCtas = 8;                           // of an SM, at least
constexpr int kGrid = 16 * kSMs;                       // CTAs of one launch at most
constexpr int kJobsMost = 1000;                        // tensors of one launch at most

struct Partial;

// One tensor.  Octets start at element `head` for the norm (a 16-byte boundary
// of src), `dst_head` for the clipping (one of dst); the elements before it
// and after the last whole octet go one by one.
struct GradJob {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t tile_begin;
  uint8_t src_type, dst_type, head, dst_head;
};
static_assert(sizeof(GradJob) == 32, "job table entries");

// Passed by value (at most 32 KB of kernel parameters), so that the table
// needs no device memory; three sizes, as a launch's cost grows with them.
template <int CAP>
struct GradArgs {
  Partial* partials;  // of every launch of the call
  zero_norm_result* result;
  float max_norm;         // negative: no factor is wanted
  int32_t n_partials;     // of every launch of the call
  int32_t partial_base;   // this launch's first partial
  int32_t n_jobs, n_tiles;
  int32_t inf_norm, leader;  // leader: this launch writes the result
  GradJob jobs[CAP];
};

// Sums of squares of binary32 values without overflow or underflow that could
// show: |g| < 2^20 goes to a as (2^20 g)^2 < 2^80, the rest to b as
// (2^-84 g)^2 < 2^88.  Both scalings are exact; no number of squares that fits
// the device overflows, values down to 2^-83 keep normal squares, an infinity
// or NaN makes its sum non-finite.  fp16 values never leave the first range.
// binary64 would need no ranges, but its units are few here: with binary64
// sums, 1500 tensors of 12M elements took 98 us to clip in place of 58, 101M
// bf16 values 119 in place of 111.
constexpr float kMidScale = 0x1p20f, kBigFrom = 0x1p20f, kBigScale = 0x1p-84f;

struct Squares {
  F2 a[2];
  float b;
};

template <class T>
__device__ __forceinline__ void add_squares(Squares& s, const float (&v)[8]) {
  if constexpr (Elem<T>::kType != ZERO_FP16) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
    if (!(m < kBigFrom)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool big = !(fabsf(v[k]) < kBigFrom);
        const float w = v[k] * (big ? kBigScale : kMidScale);
        if (big)
          s.b = fmaf(w, w, s.b);
        else
          s.a[k & 1] = fma2(f2(w, 0.f), f2(w, 0.f), s.a[k & 1]);
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const F2 w = mul2(f2(v[2 * k], v[2 * k + 1]), f2(kMidScale));
    s.a[k & 1] = fma2(w, w, s.a[k & 1]);
  }
}

// A sum held as two binary32 numbers (about 48 bits); sums of long chains of
// parts are kept this way.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair pair_add(Pair x, Pair y) {
  const float s = x.hi + y.hi;
  const float t = s - x.hi;
  const float e = (x.hi - (s - t)) + (y.hi - t) + (x.lo + y.lo);
  // an infinity or NaN stays what it is
  if (!(fabsf(s) < INFINITY)) return {s, 0.f};
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
__device__ __forceinline__ Pair pair_xor(Pair x, int o) {
  return {__shfl_xor_sync(kFull, x.hi, o), __shfl_xor_sync(kFull, x.lo, o)};
}

// What a CTA leaves: its sums, or the largest |g| as a's hi.
struct alignas(16) Partial {
  Pair a, b;
};

// The bits of |g| order as unsigned integers, NaN above infinity.
__device__ __forceinline__ void add_max(uint32_t& m, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
}

__device__ __forceinline__ float bits_max(float x, float y) {  // of magnitudes, NaN above all
  return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
}

__device__ __forceinline__ Partial join(Partial x, const Partial& y, bool inf_norm) {
  if (inf_norm) {
    x.a.hi = bits_max(x.a.hi, y.a.hi);
  } else {
    x.a = pair_add(x.a, y.a);
    x.b = pair_add(x.b, y.b);
  }
  return x;
}

// The CTA's partial from its threads', in a fixed order; the same in every thread.
__device__ __forceinline__ Partial block_join(Partial x, bool inf_norm, Partial* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = join(x, Partial{pair_xor(x.a, o), pair_xor(x.b, o)}, inf_norm);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int w = 1; w < kNormThreads / 32; ++w) x = join(x, part[w], inf_norm);
  __syncthreads();
  return x;
}

template <int CAP>
__device__ __forceinline__ int find_grad_job(const GradArgs<CAP>& a, int tile) {
  int lo = 0, hi = a.n_jobs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.jobs[mid].tile_begin <= tile)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// An octet from an address off the 16-byte boundaries: the covering chunks,
// shifted by whole words and, for 16-bit elements, by half a word.  All chunks
// lie in the tensor.
template <class T>
__device__ __forceinline__ void load_shifted(Octet<T>& o, const T* p) {
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - skip);
  uint32_t x[4 * Octet<T>::kChunks + 5];
#pragma unroll
  for (int k = 0; k <= Octet<T>::kChunks; ++k) {
    const uint4 c = __ldg(q + k);
    x[4 * k] = c.x, x[4 * k + 1] = c.y, x[4 * k + 2] = c.z, x[4 * k + 3] = c.w;
  }
  x[4 * Octet<T>::kChunks + 4] = 0;
  uint32_t y[4 * Octet<T>::kChunks + 1];
#pragma unroll
  for (int k = 0; k <= 4 * Octet<T>::kChunks; ++k) {  // a word more than the octet's, for the half shift
    const uint32_t lo = skip & 4 ? x[k + 1] : x[k];
    const uint32_t hi = k + 3 < 4 * Octet<T>::kChunks + 5 ? (skip & 4 ? x[k + 3] : x[k + 2]) : 0;
    y[k] = skip & 8 ? hi : lo;
  }
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < 4 * Octet<T>::kChunks; ++k) y[k] = __funnelshift_r(y[k], y[k + 1], 8 * (skip & 2));
  }
#pragma unroll
  for (int k = 0; k < Octet<T>::kChunks; ++k)
    o.w[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
}

// Elements [e0, e0 + cnt) of a tensor, one by one, zero elsewhere.
template <class T>
__device__ __forceinline__ void load_some(const T* src, int e0, int cnt, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < cnt ? Elem<T>::widen(src[e0 + k]) : 0.f;
}

// A tile of a tensor in its own elements: octets lie at 8 * thread + 1024 k,
// elements [0, left) exist.  The tile of element 0 has `before` elements in
// front, down to the tensor's start.
struct Tile {
  int64_t base;
  int left, before;
  __device__ __forceinline__ Tile(const GradJob& j, int head, int t) {
    base = head + static_cast<int64_t>(t) * kNormTile;
    left = static_cast<int>(max(static_cast<int64_t>(-1), min(j.numel - base, static_cast<int64_t>(kNormTile + 64))));
    before = t == 0 ? static_cast<int>(min(static_cast<int64_t>(head), j.numel)) : kNormTile;
  }
  static __device__ __forceinline__ int at(int k) { return (k * kNormThreads + static_cast<int>(threadIdx.x)) * 8; }
};

// The octets of a tile that is not whole, two at a time: octets(e, f) for whole
// ones (f -1: one only), some(e, cnt) for single elements, e relative to the
// tile.  good(e): the octet at e may be taken whole.
template <class Good, class Two, class Some>
__device__ __forceinline__ void part_of_tile(const Tile& tile, int t, Good good, Two octets, Some some) {
  if (t == 0 && threadIdx.x == 0 && tile.before > 0) some(-static_cast<int>(tile.base), tile.before);
#pragma unroll 1
  for (int e = Tile::at(0); e < min(tile.left, kNormTile); e += 2 * kNormThreads * 8) {
    const int f = e + kNormThreads * 8;
    if (good(e) && good(f) && f < kNormTile) {
      octets(e, f);
      continue;
    }
#pragma unroll 1
    for (int x = e; x < min(tile.left, min(f + 1, kNormTile)); x += kNormThreads * 8) {
      if (good(x))
        octets(x, -1);
      else
        some(x, min(8, tile.left - x));
    }
  }
}

template <class T>
__device__ __forceinline__ void norm_tile(const GradJob& j, int t, bool inf_norm, Squares& s, uint32_t& m) {
  const Tile tile(j, j.head, t);
  const T* src = static_cast<const T*>(j.src) + tile.base;
  auto take = [&](const float (&v)[8]) {
    if (inf_norm)
      add_max(m, v);
    else
      add_squares<T>(s, v);
  };
  if (tile.left >= kNormTile && (t > 0 || j.head == 0)) {
    constexpr int kTogether = kBytesAhead / 8 / sizeof(T);
#pragma unroll
    for (int k0 = 0; k0 < kAhead; k0 += kTogether) {
      Octet<T> o[kTogether];
#pragma unroll
      for (int k = 0; k < kTogether; ++k) o[k].load(src + Tile::at(k0 + k));
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        float v[8];
        o[k].widen(v);
        take(v);
      }
    }
    return;
  }
  part_of_tile(
      tile, t, [&](int e) { return e + 8 <= tile.left; },
      [&](int e, int f) {
        Octet<T> o, p;
        o.load(src + e);
        if (f >= 0) p.load(src + f);
        float v[8];
        o.widen(v);
        take(v);
        if (f >= 0) {
          p.widen(v);
          take(v);
        }
      },
      [&](int e, int cnt) {
        float v[8];
        load_some(src, e, cnt, v);
        take(v);
      });
}

// 212M fp32 values in 126 us (0.99 of a plain copy's bandwidth), bf16 in 70
// (0.89); 1M values: two launches' latency.
template <int CAP>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) k_grad_norm(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ Partial part[kNormThreads / 32];
  let_next_start();
  const int lo = static_cast<int>(static_cast<int64_t>(a.n_tiles) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(a.n_tiles) * (blockIdx.x + 1) / gridDim.x);
  const bool inf_norm = a.inf_norm != 0;
  Partial sum = {{0.f, 0.f}, {0.f, 0.f}};
  Squares s = {{f2(0.f), f2(0.f)}, 0.f};
  uint32_t m = 0;
  int q = find_grad_job(a, lo);
  for (int tile = lo; tile < hi; ++tile) {
    while (q + 1 < a.n_jobs && a.jobs[q + 1].tile_begin <= tile) ++q;
    const GradJob& j = a.jobs[q];
    const int t = tile - j.tile_begin;
    if (j.src_type == ZERO_FP32)
      norm_tile<float>(j, t, inf_norm, s, m);
    else if (j.src_type == ZERO_BF16)
      norm_tile<__nv_bfloat16>(j, t, inf_norm, s, m);
    else
      norm_tile<__half>(j, t, inf_norm, s, m);
    // a thread has at most 71 squares of a tile before they join a pair: all of
    // them in one binary32 sum where values of the upper range take part, 20
    // in each of four otherwise
    sum.a = pair_add(sum.a, {sum2(add2(s.a[0], s.a[1])), 0.f});
    if (s.b != 0.f) sum.b = pair_add(sum.b, {s.b, 0.f});
    s = {{f2(0.f), f2(0.f)}, 0.f};
  }
  if (inf_norm) sum.a.hi = __uint_as_float(m);
  sum = block_join(sum, inf_norm, part);
  if (threadIdx.x == 0) a.partials[a.partial_base + blockIdx.x] = sum;
}

// The factor from every partial of the call, the same in every CTA, in
// binary32; the leader's first CTA writes the record.
template <int CAP>
__device__ __forceinline__ float decide(const GradArgs<CAP>& a, Partial* part) {
  const bool inf_norm = a.inf_norm != 0;
  wait_for_previous();
  Partial x = {{0.f, 0.f}, {0.f, 0.f}};
  for (int p = threadIdx.x; p < a.n_partials; p += 4 * kNormThreads) {
    float4 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = p + k * kNormThreads < a.n_partials
                 ? __ldcg(reinterpret_cast<const float4*>(a.partials) + p + k * kNormThreads)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) x = join(x, Partial{{y[k].x, y[k].y}, {y[k].z, y[k].w}}, inf_norm);
  }
  x = block_join(x, inf_norm, part);
  // the norm times `unit`, which keeps it in range: the sum of two ranges'
  // squares is that of the larger one's, the other's scaled to it
  float norm, unit = 1.f;
  if (inf_norm) {
    norm = x.a.hi;
  } else if (x.b.hi == 0.f) {
    norm = sqrtf(x.a.hi) * 0x1p-20f;
  } else {
    norm = sqrtf(x.b.hi + x.a.hi * 0x1p-104f * 0x1p-104f) * 0x1p20f;
    unit = 0x1p-64f;
  }
  const bool fine = norm < INFINITY;
  float coef = 1.f;
  if (fine && a.max_norm >= 0.f) coef = fminf(1.f, a.max_norm * unit / (norm + 1e-6f * unit));
  if (a.leader && blockIdx.x == 0 && threadIdx.x == 0) {
    zero_norm_result r = {};
    if (inf_norm)
      r.norm = x.a.hi;
    else
      r.norm = sqrt((static_cast<double>(x.a.hi) + x.a.lo) * 0x1p-40 +
                    (static_cast<double>(x.b.hi) + x.b.lo) * 0x1p168);
    r.norm32 = static_cast<float>(r.norm);
    r.coef = coef;
    r.nonfinite = fine ? 0 : 1;
    *a.result = r;
  }
  return coef;
}

template <int CAP>
__global__ void __launch_bounds__(kNormThreads) k_norm_result(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ Partial part[kNormThreads / 32];
  decide(a, part);
}

// An octet to a 16-byte boundary, not kept in L2: nothing here reads it.
template <class D>
__device__ __forceinline__ void store_octet(D* p, const float (&v)[8]) {
  if constexpr (sizeof(D) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(Elem<D>::pack(v[0], v[1]), Elem<D>::pack(v[2], v[3]),
                                                   Elem<D>::pack(v[4], v[5]), Elem<D>::pack(v[6], v[7])));
  }
}

template <class S, class D>
__device__ __forceinline__ void clip_tile(const GradJob& j, int t, float coef) {
  const Tile tile(j, j.dst_head, t);
  const S* src = static_cast<const S*>(j.src) + tile.base;
  D* dst = static_cast<D*>(j.dst) + tile.base;
  // octets lie on dst's boundaries; src's then lie there too or all off by as
  // much, and the chunks of those at either end of the tensor reach past it
  const bool straight = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  auto scaled = [&](const Octet<S>& o, int e) {
    float v[8];
    o.widen(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= coef;
    store_octet(dst + e, v);
  };
  if (tile.left >= kNormTile + 16 && t > 0) {
    if (straight) {
      constexpr int kTogether = kBytesAhead / 8 / sizeof(S);
#pragma unroll
      for (int k0 = 0; k0 < kAhead; k0 += kTogether) {
        Octet<S> o[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) o[k].load(src + Tile::at(k0 + k));
#pragma unroll
        for (int k = 0; k < kTogether; ++k) scaled(o[k], Tile::at(k0 + k));
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < kAhead; k += 2) {
        Octet<S> o[2];
        load_shifted(o[0], src + Tile::at(k));
        load_shifted(o[1], src + Tile::at(k + 1));
        scaled(o[0], Tile::at(k));
        scaled(o[1], Tile::at(k + 1));
      }
    }
    return;
  }
  part_of_tile(
      tile, t,
      [&](int e) { return straight ? e + 8 <= tile.left : e + tile.before >= 8 && e + 16 <= tile.left; },
      [&](int e, int f) {
        Octet<S> o, p;
        if (straight) {
          o.load(src + e);
          if (f >= 0) p.load(src + f);
        } else {
          load_shifted(o, src + e);
          if (f >= 0) load_shifted(p, src + f);
        }
        scaled(o, e);
        if (f >= 0) scaled(p, f);
      },
      [&](int e, int cnt) {
        float v[8];
        load_some(src, e, cnt, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cnt) dst[e + k] = Elem<D>::narrow(v[k] * coef);
      });
}

template <class S>
__device__ __forceinline__ void clip_tile_to(const GradJob& j, int t, float coef) {
  if (j.dst_type == ZERO_FP32)
    clip_tile<S, float>(j, t, coef);
  else if (j.dst_type == ZERO_BF16)
    clip_tile<S, __nv_bfloat16>(j, t, coef);
  else
    clip_tile<S, __half>(j, t, coef);
}

// Norm and clipping of 101M bf16 values into a replica: 101-106 us, of which the
// norm's pass 36; 74 would be every second read from L2.
template <int CAP>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) k_grad_clip(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ Partial part[kNormThreads / 32];
  const float coef = decide(a, part);
  // the last CTAs' tiles first: the norm read them last
  const int block = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  const int lo = static_cast<int>(static_cast<int64_t>(a.n_tiles) * block / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(a.n_tiles) * (block + 1) / gridDim.x);
  int q = find_grad_job(a, hi > lo ? hi - 1 : lo);
  for (int tile = hi - 1; tile >= lo; --tile) {
    while (a.jobs[q].tile_begin > tile) --q;
    const GradJob& j = a.jobs[q];
    if (coef == 1.f && j.src == j.dst) continue;  // in place and nothing to scale
    const int t = tile - j.tile_begin;
    if (j.src_type == ZERO_FP32)
      clip_tile_to<float>(j, t, coef);
    else if (j.src_type == ZERO_BF16)
      clip_tile_to<__nv_bfloat16>(j, t, coef);
    else
      clip_tile_to<__half>(j, t, coef);
  }
}

// ---------------------------------------------------------------------------
// host

struct Batch {  // the tensors of one launch
  std::vector<GradJob> jobs;
  int64_t tiles = 0;
  int grid() const { return static_cast<int>(std::min<int64_t>(tiles, kGrid)); }
};

struct Call {
  std::vector<Batch> batches;
  double max_norm = -1.0;
  bool inf_norm = false;
  zero_norm_result* result = nullptr;
  Partial* partials = nullptr;
  int n_partials = 0;
  cudaStream_t stream = nullptr;
};

enum class Pass { kNorm, kClip, kResult };

template <int CAP>
int launch_pass(const Call& c, const Batch* b, int base, bool leader, bool early, Pass pass) {
  auto* a = new (std::nothrow) GradArgs<CAP>();
  if (!a) return static_cast<int>(cudaErrorMemoryAllocation);
  a->partials = c.partials;
  a->result = c.result;
  a->max_norm = static_cast<float>(c.max_norm);
  a->n_partials = c.n_partials;
  a->partial_base = base;
  a->inf_norm = c.inf_norm;
  a->leader = leader;
  int grid = 1;
  if (b) {
    a->n_jobs = static_cast<int32_t>(b->jobs.size());
    a->n_tiles = static_cast<int32_t>(b->tiles);
    std::copy(b->jobs.begin(), b->jobs.end(), a->jobs);
    grid = b->grid();
  }
  void* args[] = {a};
  const void* fn = pass == Pass::kNorm   ? reinterpret_cast<const void*>(&k_grad_norm<CAP>)
                   : pass == Pass::kClip ? reinterpret_cast<const void*>(&k_grad_clip<CAP>)
                                         : reinterpret_cast<const void*>(&k_norm_result<CAP>);
  const cudaError_t e = launch_maybe_early(fn, dim3(grid), dim3(kNormThreads), args, early, c.stream);
  delete a;
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return static_cast<int>(e);
}

int launch_sized(const Call& c, const Batch* b, int base, bool leader, bool early, Pass pass) {
  const size_t n = b ? b->jobs.size() : 0;
  if (n <= 64) return launch_pass<64>(c, b, base, leader, early, pass);
  if (n <= 256) return launch_pass<256>(c, b, base, leader, early, pass);
  return launch_pass<kJobsMost>(c, b, base, leader, early, pass);
}

// Elements before the first 16-byte boundary.
int head_of(const void* p, int type) {
  return static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16) / type_bytes(type);
}

int64_t tiles_of(const zero_grad_tensor& t, int head) {
  const int64_t body = t.numel > head ? t.numel - head : 0;
  return std::max<int64_t>(1, (body + kNormTile - 1) / kNormTile);
}

zero_status check_list(const char* fn, const zero_grad_tensor* t, int32_t n, bool clip) {
  if (n < 0) return fail(ZERO_ERR_INVALID, "%s: n_tensors is negative", fn);
  if (n > 0 && !t) return fail(ZERO_ERR_INVALID, "%s: tensors is NULL", fn);
  for (int32_t k = 0; k < n; ++k) {
    if (t[k].numel < 0) return fail(ZERO_ERR_INVALID, "%s: tensors[%d].numel is negative", fn, k);
    if (t[k].numel > INT64_C(1) << 40)
      return fail(ZERO_ERR_INVALID, "%s: tensors[%d].numel is above 2^40", fn, k);
    if (!known_type(t[k].src_dtype))
      return fail(ZERO_ERR_INVALID, "%s: tensors[%d]: unknown src_dtype", fn, k);
    if (clip && !known_type(t[k].dst_dtype))
      return fail(ZERO_ERR_INVALID, "%s: tensors[%d]: unknown dst_dtype", fn, k);
    if (t[k].numel == 0) continue;
    if (!t[k].src) return fail(ZERO_ERR_INVALID, "%s: tensors[%d].src is NULL", fn, k);
    if (!aligned_to(t[k].src, type_bytes(t[k].src_dtype)))
      return fail(ZERO_ERR_ALIGN, "%s: tensors[%d].src is not aligned to its elements", fn, k);
    if (!clip) continue;
    if (!t[k].dst) return fail(ZERO_ERR_INVALID, "%s: tensors[%d].dst is NULL", fn, k);
    if (!aligned_to(t[k].dst, type_bytes(t[k].dst_dtype)))
      return fail(ZERO_ERR_ALIGN, "%s: tensors[%d].dst is not aligned to its elements", fn, k);
    if (t[k].src == t[k].dst && t[k].src_dtype != t[k].dst_dtype)
      return fail(ZERO_ERR_INVALID, "%s: tensors[%d] is clipped in place but its types differ", fn, k);
  }
  return ZERO_OK;
}

int64_t workspace_bytes(const zero_grad_tensor* t, int32_t n) {
  int64_t kept = 0;
  for (int32_t k = 0; k < n; ++k) kept += t[k].numel > 0;
  return std::max<int64_t>(1, (kept + kJobsMost - 1) / kJobsMost) * kGrid * static_cast<int64_t>(sizeof(Partial));
}

zero_status norm_call(const char* fn, const zero_grad_tensor* t, int32_t n, int32_t kind, bool clip,
                      double max_norm, void* d_result, void* workspace, int64_t ws_bytes,
                      void* stream) {
  clear_error();
  NvtxRange range(fn);
  if (kind != ZERO_NORM_L2 && kind != ZERO_NORM_INF)
    return fail(ZERO_ERR_INVALID, "%s: kind must be ZERO_NORM_L2 or ZERO_NORM_INF", fn);
  if (clip && !(isfinite(max_norm) && max_norm >= 0.0))
    return fail(ZERO_ERR_INVALID, "%s: max_norm must be finite and >= 0", fn);
  const zero_status st = check_list(fn, t, n, clip);
  if (st != ZERO_OK) return st;
  if (!d_result) return fail(ZERO_ERR_INVALID, "%s: d_result is NULL", fn);
  if (!workspace) return fail(ZERO_ERR_INVALID, "%s: workspace is NULL", fn);
  if (!aligned_to(d_result, 16) || !aligned_to(workspace, 16))
    return fail(ZERO_ERR_ALIGN, "%s: d_result and workspace must be 16-byte aligned", fn);
  const int64_t need = workspace_bytes(t, n);
  if (ws_bytes < need)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, ws_bytes, need);
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));

  Call c;
  c.max_norm = clip ? max_norm : -1.0;
  c.inf_norm = kind == ZERO_NORM_INF;
  c.result = static_cast<zero_norm_result*>(d_result);
  c.partials = static_cast<Partial*>(workspace);
  c.stream = static_cast<cudaStream_t>(stream);
  try {
    for (int32_t k = 0; k < n; ++k) {
      if (t[k].numel == 0) continue;
      if (c.batches.empty() || c.batches.back().jobs.size() == kJobsMost) c.batches.emplace_back();
      Batch& b = c.batches.back();
      GradJob j = {};
      j.src = t[k].src;
      j.dst = clip ? t[k].dst : nullptr;
      j.numel = t[k].numel;
      j.tile_begin = static_cast<int32_t>(b.tiles);
      j.src_type = static_cast<uint8_t>(t[k].src_dtype);
      j.dst_type = static_cast<uint8_t>(clip ? t[k].dst_dtype : t[k].src_dtype);
      const int head = head_of(j.src, j.src_type), dst_head = clip ? head_of(j.dst, j.dst_type) : head;
      j.head = static_cast<uint8_t>(head);
      j.dst_head = static_cast<uint8_t>(dst_head);
      b.jobs.push_back(j);
      b.tiles += tiles_of(t[k], std::min(head, dst_head));  // enough for either pass
      if (b.tiles > INT32_MAX / 2)
        return fail(ZERO_ERR_INVALID, "%s: the tensors hold too many elements for one call", fn);
    }
  } catch (const std::bad_alloc&) {
    return fail(ZERO_ERR_OOM, "%s: out of host memory", fn);
  }
  for (const Batch& b : c.batches) c.n_partials += b.grid();
  int e = 0, base = 0;
  for (const Batch& b : c.batches) {
    if (!e) e = launch_sized(c, &b, base, false, false, Pass::kNorm);
    base += b.grid();
  }
  // The first launch after the norm's starts early: it waits for them on the
  // device.  (A further launch of the clipping is an ordinary one.)
  const bool one = !c.batches.empty();
  if (!clip || c.batches.empty()) {
    if (!e) e = launch_sized(c, nullptr, 0, true, one, Pass::kResult);
  } else {
    const size_t last = c.batches.size() - 1;
    for (size_t k = last + 1; k-- > 0;)
      if (!e) e = launch_sized(c, &c.batches[k], 0, k == last, k == last, Pass::kClip);
  }
  if (e)
    return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(static_cast<cudaError_t>(e)));
  return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_grad_norm_workspace_bytes(const zero_grad_tensor* tensors, int32_t n_tensors,
                                                      int64_t* bytes) {
  clear_error();
  const char* fn = "zero_grad_norm_workspace_bytes";
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  const zero_status st = check_list(fn, tensors, n_tensors, false);
  if (st != ZERO_OK) return st;
  *bytes = workspace_bytes(tensors, n_tensors);
  return ZERO_OK;
}

extern "C" zero_status zero_grad_norm(const zero_grad_tensor* tensors, int32_t n_tensors, int32_t kind,
                                      void* d_result, void* workspace, int64_t workspace_bytes_,
                                      void* stream) {
  return norm_call("zero_grad_norm", tensors, n_tensors, kind, false, 0.0, d_result, workspace,
                   workspace_bytes_, stream);
}

extern "C" zero_status zero_clip_grad_norm(const zero_grad_tensor* tensors, int32_t n_tensors,
                                           int32_t kind, double max_norm, void* d_result,
                                           void* workspace, int64_t workspace_bytes_, void* stream) {
  return norm_call("zero_clip_grad_norm", tensors, n_tensors, kind, true, max_norm, d_result, workspace,
                   workspace_bytes_, stream);
}
