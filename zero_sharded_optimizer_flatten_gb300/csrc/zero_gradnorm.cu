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
// Work split: a tensor is cut into tiles of 4096 elements, a CTA takes a
// contiguous run of tiles (of any tensors) and leaves one binary64 partial,
// so the partials are few (at most kGrid a launch) and every CTA of the
// clipping adds them up itself, in the same fixed order: no kernel between
// the two passes, no atomics, the same norm in every run.  The clipping walks
// the tiles from the last to the first, so what the norm read last is still
// in L2.
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

constexpr int kNormThreads = 256;
constexpr int kNormTile = 4096;                        // elements a CTA takes at once
constexpr int kTileOctets = kNormTile / 8;             // 512: two octets a thread
constexpr int kGrid = 8 * kSMs;                        // CTAs of one launch at most
constexpr int kJobsMost = 1000;                        // tensors of one launch at most

// One tensor.  head: elements before the first 16-byte boundary of src (they
// go one by one, as do the elements after the last whole octet).
struct GradJob {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t tile_begin;
  uint8_t src_type, dst_type, head, vec_store;
};
static_assert(sizeof(GradJob) == 32, "job table entries");

// Passed by value (at most 32 KB of kernel parameters), so that the table
// needs no device memory; three sizes, as a launch's cost grows with them.
template <int CAP>
struct GradArgs {
  double* partials;       // of every launch of the call
  zero_norm_result* result;
  double max_norm;
  int32_t n_partials;     // of every launch of the call
  int32_t partial_base;   // this launch's first partial
  int32_t n_jobs, n_tiles;
  int32_t inf_norm, leader;  // leader: this launch writes the result
  GradJob jobs[CAP];
};

// Squares of binary32 values without overflow or underflow that could show:
// |g| < 2^20 goes to a as (2^40 g)^2, the rest to b as (2^-68 g)^2.  Both
// scalings are exact; 64 squares of either range stay finite, values down to
// 2^-103 keep normal squares, an infinity or NaN makes its sum non-finite.
// fp16 values never leave the first range.
struct Squares {
  float a[2], b;
};

template <class T>
__device__ __forceinline__ void add_squares(Squares& s, const float (&v)[8]) {
  if constexpr (Elem<T>::kType != ZERO_FP16) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
    if (!(m < 0x1p20f)) {
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        if (fabsf(v[k]) < 0x1p20f)
          s.a[0] = fmaf(v[k] * 0x1p40f, v[k] * 0x1p40f, s.a[0]);
        else
          s.b = fmaf(v[k] * 0x1p-68f, v[k] * 0x1p-68f, s.b);
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float w = v[k] * 0x1p40f;
    s.a[k & 1] = fmaf(w, w, s.a[k & 1]);
  }
}

// The bits of |g| order as unsigned integers, NaN above infinity.
__device__ __forceinline__ void add_max(uint32_t& m, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
}

__device__ __forceinline__ double nan_max(double x, double y) {
  return x != x || y != y ? x + y : fmax(x, y);
}

// The CTA's sum (or maximum) of one binary64 value a thread, in a fixed
// order; the same value in every thread.
__device__ __forceinline__ double block_join(double x, bool inf_norm, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double y = __shfl_xor_sync(kFull, x, o);
    x = inf_norm ? nan_max(x, y) : x + y;
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double t = part[0];
#pragma unroll
  for (int w = 1; w < kNormThreads / 32; ++w) t = inf_norm ? nan_max(t, part[w]) : t + part[w];
  __syncthreads();
  return t;
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

// Elements [e0, e0 + cnt) of a tensor, zero elsewhere.
template <class T>
__device__ __forceinline__ void load_octet(const T* src, int64_t e0, int cnt, float (&v)[8]) {
  if (cnt == 8) {
    Elem<T>::load8(src + e0, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < cnt ? Elem<T>::widen(src[e0 + k]) : 0.f;
  }
}

// Calls body(e0, cnt) for the thread's octets of tile `t` of a tensor: whole
// octets start at element `head`; the elements before it are an octet of
// their own, of the first tile's thread 0.
template <class Body>
__device__ __forceinline__ void for_octets(const GradJob& j, int t, Body body) {
  if (t == 0 && threadIdx.x == 0 && j.head)
    body(static_cast<int64_t>(0), static_cast<int>(min(static_cast<int64_t>(j.head), j.numel)));
#pragma unroll
  for (int k = 0; k < kTileOctets / kNormThreads; ++k) {
    const int64_t e0 = j.head + (static_cast<int64_t>(t) * kTileOctets + k * kNormThreads + threadIdx.x) * 8;
    if (e0 < j.numel) body(e0, static_cast<int>(min(static_cast<int64_t>(8), j.numel - e0)));
  }
}

template <class T>
__device__ __forceinline__ void norm_tile(const GradJob& j, int t, bool inf_norm, Squares& s, uint32_t& m) {
  const T* src = static_cast<const T*>(j.src);
  for_octets(j, t, [&](int64_t e0, int cnt) {
    float v[8];
    load_octet(src, e0, cnt, v);
    if (inf_norm)
      add_max(m, v);
    else
      add_squares<T>(s, v);
  });
}

template <int CAP>
__global__ void __launch_bounds__(kNormThreads) k_grad_norm(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ double part[kNormThreads / 32];
  const int lo = static_cast<int>(static_cast<int64_t>(a.n_tiles) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(a.n_tiles) * (blockIdx.x + 1) / gridDim.x);
  const bool inf_norm = a.inf_norm != 0;
  double sum = 0.0;
  uint32_t m = 0;
  Squares s = {{0.f, 0.f}, 0.f};
  int held = 0;
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
    // at most 3 tiles of up to 17..24 squares in binary32 before they join
    // the binary64 sum (head octets included: 3 * 24 = 72 squares over three
    // accumulators, none above 64)
    if (++held == 3 || tile + 1 == hi) {
      sum += static_cast<double>(s.a[0] + s.a[1]) * 0x1p-80;
      if (s.b != 0.f) sum += static_cast<double>(s.b) * 0x1p136;
      s = {{0.f, 0.f}, 0.f};
      held = 0;
    }
  }
  if (inf_norm) sum = static_cast<double>(__uint_as_float(m));
  sum = block_join(sum, inf_norm, part);
  if (threadIdx.x == 0) a.partials[a.partial_base + blockIdx.x] = sum;
}

// The norm from every partial of the call, the same in every CTA, and the
// factor; the leader's first CTA writes the record.
template <int CAP>
__device__ __forceinline__ float decide(const GradArgs<CAP>& a, double* part) {
  const bool inf_norm = a.inf_norm != 0;
  double x = 0.0;
  for (int p = threadIdx.x; p < a.n_partials; p += kNormThreads) {
    const double y = __ldcg(a.partials + p);
    x = inf_norm ? nan_max(x, y) : x + y;
  }
  x = block_join(x, inf_norm, part);
  const double norm = inf_norm ? x : sqrt(x);
  const bool fine = isfinite(norm);
  double c = 1.0;
  if (fine && a.max_norm >= 0.0) {
    const double f = a.max_norm / (norm + 1e-6);
    if (f < 1.0) c = f;
  }
  const float coef = static_cast<float>(c);
  if (a.leader && blockIdx.x == 0 && threadIdx.x == 0) {
    zero_norm_result r = {};
    r.norm = norm;
    r.norm32 = static_cast<float>(norm);
    r.coef = coef;
    r.nonfinite = fine ? 0 : 1;
    *a.result = r;
  }
  return coef;
}

template <int CAP>
__global__ void __launch_bounds__(kNormThreads) k_norm_result(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ double part[kNormThreads / 32];
  decide(a, part);
}

template <class S, class D>
__device__ __forceinline__ void clip_tile(const GradJob& j, int t, float coef) {
  const S* src = static_cast<const S*>(j.src);
  D* dst = static_cast<D*>(j.dst);
  const bool vec = j.vec_store != 0;
  for_octets(j, t, [&](int64_t e0, int cnt) {
    float v[8];
    load_octet(src, e0, cnt, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= coef;
    if (cnt == 8 && vec) {
      Elem<D>::store8(dst + e0, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < cnt) dst[e0 + k] = Elem<D>::narrow(v[k]);
    }
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

template <int CAP>
__global__ void __launch_bounds__(kNormThreads) k_grad_clip(const __grid_constant__ GradArgs<CAP> a) {
  __shared__ double part[kNormThreads / 32];
  const float coef = decide(a, part);
  const int lo = static_cast<int>(static_cast<int64_t>(a.n_tiles) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(a.n_tiles) * (blockIdx.x + 1) / gridDim.x);
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
  double* partials = nullptr;
  int n_partials = 0;
  cudaStream_t stream = nullptr;
};

enum class Pass { kNorm, kClip, kResult };

template <int CAP>
int launch_pass(const Call& c, const Batch* b, int base, bool leader, Pass pass) {
  auto* a = new (std::nothrow) GradArgs<CAP>();
  if (!a) return static_cast<int>(cudaErrorMemoryAllocation);
  a->partials = c.partials;
  a->result = c.result;
  a->max_norm = c.max_norm;
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
  const cudaError_t e = cudaLaunchKernel(fn, dim3(grid), dim3(kNormThreads), args, 0, c.stream);
  delete a;
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return static_cast<int>(e);
}

int launch_sized(const Call& c, const Batch* b, int base, bool leader, Pass pass) {
  const size_t n = b ? b->jobs.size() : 0;
  if (n <= 64) return launch_pass<64>(c, b, base, leader, pass);
  if (n <= 256) return launch_pass<256>(c, b, base, leader, pass);
  return launch_pass<kJobsMost>(c, b, base, leader, pass);
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
  return std::max<int64_t>(1, (kept + kJobsMost - 1) / kJobsMost) * kGrid * static_cast<int64_t>(sizeof(double));
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
  c.partials = static_cast<double*>(workspace);
  c.stream = static_cast<cudaStream_t>(stream);
  try {
    for (int32_t k = 0; k < n; ++k) {
      if (t[k].numel == 0) continue;
      if (c.batches.empty() || c.batches.back().jobs.size() == kJobsMost) c.batches.emplace_back();
      Batch& b = c.batches.back();
      const int sb = type_bytes(t[k].src_dtype);
      const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(t[k].src) & 15)) % 16) / sb;
      GradJob j = {};
      j.src = t[k].src;
      j.dst = clip ? t[k].dst : nullptr;
      j.numel = t[k].numel;
      j.tile_begin = static_cast<int32_t>(b.tiles);
      j.src_type = static_cast<uint8_t>(t[k].src_dtype);
      j.dst_type = static_cast<uint8_t>(clip ? t[k].dst_dtype : t[k].src_dtype);
      j.head = static_cast<uint8_t>(head);
      j.vec_store = clip && aligned_to(static_cast<char*>(t[k].dst) + head * type_bytes(t[k].dst_dtype), 16);
      b.jobs.push_back(j);
      b.tiles += tiles_of(t[k], head);
      if (b.tiles > INT32_MAX / 2)
        return fail(ZERO_ERR_INVALID, "%s: the tensors hold too many elements for one call", fn);
    }
  } catch (const std::bad_alloc&) {
    return fail(ZERO_ERR_OOM, "%s: out of host memory", fn);
  }
  for (const Batch& b : c.batches) c.n_partials += b.grid();
  int e = 0, base = 0;
  for (const Batch& b : c.batches) {
    if (!e) e = launch_sized(c, &b, base, false, Pass::kNorm);
    base += b.grid();
  }
  if (!clip || c.batches.empty()) {
    if (!e) e = launch_sized(c, nullptr, 0, true, Pass::kResult);
  } else {
    for (size_t k = c.batches.size(); k-- > 0;)
      if (!e) e = launch_sized(c, &c.batches[k], 0, k == 0, Pass::kClip);
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
