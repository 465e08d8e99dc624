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
#include "zero_rows.cuh"

namespace cg = cooperative_groups;

namespace zero {
namespace {

// ---------------------------------------------------------------------------
// The sort: a stable counting sort by one thread-block cluster.  The pairs
// are cut into one contiguous segment a warp; a warp counts its segment's
// experts in its own shared-memory row, the rows are scanned across the
// cluster's warps (through distributed shared memory) and the experts, and
// the warp walks its segment again giving out places.  Lanes with the same
// expert find their rank by a warp match, so the order is stable and nothing
// depends on timing.
//
// One launch and no global scratch.  It is bound by the walk's latency
// (32 pairs a step and warp), not by bytes: a cluster of up to kSortCtas
// CTAs shortens the segments.

constexpr int kSortCtas = 8;           // CTAs of the largest cluster (portable size)
constexpr int kSortWarpsMost = 32;
constexpr int kMaxExperts = 4096;
constexpr int kSortSmemMost = 200 * 1024;

struct SortArgs {
  const void* ids;
  int64_t n;           // pairs
  int32_t id_bytes, n_experts;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pairs;
};

__device__ __forceinline__ int load_id(const SortArgs& a, int64_t p) {
  if (a.id_bytes == 4) {
    const int v = static_cast<const int*>(a.ids)[p];
    return v >= 0 && v < a.n_experts ? v : -1;
  }
  const long long v = static_cast<const long long*>(a.ids)[p];
  return v >= 0 && v < a.n_experts ? static_cast<int>(v) : -1;
}

__global__ void __launch_bounds__(32 * kSortWarpsMost) k_expert_sort(const SortArgs a) {
  extern __shared__ int smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int E = a.n_experts;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
  int* count = smem;               // [warps][E]
  int* total = smem + warps * E;   // [E]: this CTA's pairs of each expert
  int* start = total + E;          // [E]: first row of each expert for this CTA
  int* scan = start + E;           // [warps]
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  // this warp's pairs: whole groups of 32 but for the last warp
  const int64_t all = static_cast<int64_t>(ctas) * warps;
  const int64_t seg = (((a.n + all - 1) / all) + 31) / 32 * 32;
  const int64_t lo = min(a.n, (static_cast<int64_t>(me) * warps + warp) * seg);
  const int64_t hi = min(a.n, lo + seg);
  int* mine = count + warp * E;
  for (int64_t p = lo; p < hi; p += 32) {
    const int e = p + lane < hi ? load_id(a, p + lane) : -1;
    const unsigned same = __match_any_sync(kFull, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
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
  cluster.sync();
  // the pairs of all CTAs below this one, and of all CTAs, expert by expert;
  // then an exclusive scan of the latter over the experts
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int below = 0, sum = 0;
    if (e < E) {
      for (int c = 0; c < ctas; ++c) {
        const int v = cluster.map_shared_rank(total, c)[e];
        if (c < me) below += v;
        sum += v;
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
  for (int64_t p = lo; p < hi; p += 32) {
    const int e = p + lane < hi ? load_id(a, p + lane) : -1;
    const unsigned same = __match_any_sync(kFull, e);
    int row = -1;
    if (e >= 0) row = mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (p + lane < hi) a.rows[p + lane] = row;
    if (row >= 0) a.pairs[row] = static_cast<int>(p + lane);
  }
  for (int64_t i = M + static_cast<int64_t>(me) * blockDim.x + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(ctas) * blockDim.x)
    a.pairs[i] = -1;
  cluster.sync();  // no CTA leaves while another may still read its totals
}

// ---------------------------------------------------------------------------
// The rows.  A group of 1, 2, 4 or 8 warps takes a token.

constexpr int kRowThreads = 256;

struct RowArgs {
  const void* in;          // x, ys, dxs or dy
  const void* ys;          // combine's gradient
  const void* weights;     // null: ones
  void* out;               // xs, y, dx or dys
  void* dweights;
  const int32_t* rows;
  const int32_t* total;    // offsets + n_experts
  int64_t tokens, hidden, stride;  // stride: of in's rows (x, dy)
  int32_t topk, weight_type;
};

// Columns of one row: octets when VEC (16-byte aligned rows), else elements.
template <class T, bool VEC>
struct Cols {
  static constexpr int kN = VEC ? 8 : 1;
  static __device__ __forceinline__ void load(const T* p, float (&v)[kN]) {
    if constexpr (VEC)
      Elem<T>::load8(p, v);
    else
      v[0] = Elem<T>::widen(*p);
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[kN]) {
    if constexpr (VEC)
      Elem<T>::store8(p, v);
    else
      *p = Elem<T>::narrow(v[0]);
  }
};

// The group's token and the thread's place in the group.
struct Place {
  int64_t token;
  int lane, size;
  __device__ __forceinline__ explicit Place(int group_warps) {
    size = 32 * group_warps;
    token = static_cast<int64_t>(blockIdx.x) * (kRowThreads / size) + threadIdx.x / size;
    lane = threadIdx.x % size;
  }
};

// Rows past the last kept pair are zero: the token's own share of them.
template <class T, bool VEC>
__device__ __forceinline__ void clear_past_end(const RowArgs& a, const Place& me, T* out) {
  constexpr int N = Cols<T, VEC>::kN;
  const int64_t M = __ldg(a.total);
  const float z[N] = {};
  for (int k = 0; k < a.topk; ++k) {
    const int64_t i = me.token * a.topk + k;
    if (i < M) continue;
    for (int64_t c = static_cast<int64_t>(me.lane) * N; c < a.hidden; c += static_cast<int64_t>(me.size) * N)
      Cols<T, VEC>::store(out + i * a.hidden + c, z);
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const RowArgs a, int group_warps) {
  constexpr int N = Cols<T, VEC>::kN;
  const Place me(group_warps);
  if (me.token >= a.tokens) return;
  const T* x = static_cast<const T*>(a.in) + me.token * a.stride;
  T* xs = static_cast<T*>(a.out);
  const int32_t* rows = a.rows + me.token * a.topk;
  for (int64_t c = static_cast<int64_t>(me.lane) * N; c < a.hidden; c += static_cast<int64_t>(me.size) * N) {
    float v[N];
    Cols<T, VEC>::load(x + c, v);
    for (int k = 0; k < a.topk; ++k) {
      const int64_t r = __ldg(rows + k);
      if (r >= 0) Cols<T, VEC>::store(xs + r * a.hidden + c, v);
    }
  }
  clear_past_end<T, VEC>(a, me, xs);
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine(const RowArgs a, int group_warps) {
  constexpr int N = Cols<T, VEC>::kN;
  const Place me(group_warps);
  if (me.token >= a.tokens) return;
  const T* in = static_cast<const T*>(a.in);
  T* y = static_cast<T*>(a.out) + me.token * a.hidden;
  const int64_t p0 = me.token * a.topk;
  for (int64_t c = static_cast<int64_t>(me.lane) * N; c < a.hidden; c += static_cast<int64_t>(me.size) * N) {
    float s[N] = {};
    for (int k = 0; k < a.topk; ++k) {
      const int64_t r = __ldg(a.rows + p0 + k);
      if (r < 0) continue;
      const float w = a.weights ? load_any(a.weights, p0 + k, a.weight_type) : 1.f;
      float v[N];
      Cols<T, VEC>::load(in + r * a.hidden + c, v);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = fmaf(w, v[i], s[i]);
    }
    Cols<T, VEC>::store(y + c, s);
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_backward(const RowArgs a, int group_warps) {
  constexpr int N = Cols<T, VEC>::kN;
  __shared__ float part[2][kRowThreads / 32];
  const Place me(group_warps);
  const bool live = me.token < a.tokens;  // every thread meets the barriers below
  const T* dy = static_cast<const T*>(a.in) + (live ? me.token : 0) * a.stride;
  const T* ys = static_cast<const T*>(a.ys);
  T* dys = static_cast<T*>(a.out);
  const int64_t p0 = (live ? me.token : 0) * a.topk;
  const int warp = threadIdx.x >> 5;
  for (int k = 0; k < a.topk; ++k) {
    const int64_t r = live ? __ldg(a.rows + p0 + k) : -1;
    float dot = 0.f;
    if (r >= 0) {
      const float w = load_any(a.weights, p0 + k, a.weight_type);
      for (int64_t c = static_cast<int64_t>(me.lane) * N; c < a.hidden;
           c += static_cast<int64_t>(me.size) * N) {
        float g[N], v[N];
        Cols<T, VEC>::load(dy + c, g);
        Cols<T, VEC>::load(ys + r * a.hidden + c, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot = fmaf(g[i], v[i], dot);
          g[i] *= w;
        }
        Cols<T, VEC>::store(dys + r * a.hidden + c, g);
      }
    }
    dot = warp_all_sum(dot);
    if (group_warps > 1) {
      float* buf = part[k & 1];  // the next choice's sums go to the other half
      if ((threadIdx.x & 31) == 0) buf[warp] = dot;
      __syncthreads();
      dot = 0.f;
      const int first = warp / group_warps * group_warps;
      for (int w = 0; w < group_warps; ++w) dot += buf[first + w];
    }
    if (live && me.lane == 0 && a.dweights) store_any(a.dweights, p0 + k, a.weight_type, dot);
  }
  if (live) clear_past_end<T, VEC>(a, me, dys);
}

// ---------------------------------------------------------------------------
// host

enum class RowOp { kDispatch, kCombine, kCombineBackward };

template <class T, bool VEC>
int launch_rows(RowOp op, const RowArgs& a, cudaStream_t s) {
  // warps of a token's group: enough for the row at one octet (element) a
  // thread, a power of two up to the CTA
  const int64_t units = VEC ? a.hidden / 8 : a.hidden;
  int gw = 1;
  while (gw < kRowThreads / 32 && static_cast<int64_t>(gw) * 32 < units) gw *= 2;
  const int64_t per_cta = kRowThreads / (32 * gw);
  const int64_t grid = (a.tokens + per_cta - 1) / per_cta;
  RowArgs copy = a;
  void* args[] = {&copy, &gw};
  const void* fn = op == RowOp::kDispatch  ? reinterpret_cast<const void*>(&k_dispatch<T, VEC>)
                   : op == RowOp::kCombine ? reinterpret_cast<const void*>(&k_combine<T, VEC>)
                                           : reinterpret_cast<const void*>(&k_combine_backward<T, VEC>);
  return static_cast<int>(cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kRowThreads), args, 0, s));
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
  if (hidden < 1 || hidden > INT32_MAX)
    return fail(ZERO_ERR_INVALID, "%s: hidden must lie in [1, 2^31-1]", fn);
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

#define EXPERT_TRY(x)               \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_expert_sort(const void* ids, int32_t id_bytes, int64_t tokens, int32_t topk,
                                        int32_t n_experts, int32_t* offsets, int32_t* rows, int32_t* pairs,
                                        void* stream) {
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
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  SortArgs a = {ids, tokens * topk, id_bytes, n_experts, offsets, rows, pairs};
  // as many warps a CTA as their counters fit, no more than there are groups
  // of 32 pairs, and CTAs until a warp has four groups
  const int64_t groups = std::max<int64_t>(1, (a.n + 31) / 32);
  int warps = kSortWarpsMost;
  while (warps > 1 && (static_cast<int64_t>(warps) + 2) * n_experts * 4 + 4 * warps > kSortSmemMost) warps /= 2;
  while (warps > 1 && warps / 2 >= groups) warps /= 2;
  int ctas = 1;
  while (ctas < kSortCtas && static_cast<int64_t>(ctas) * warps * 4 < groups) ctas *= 2;
  const int smem = ((warps + 2) * n_experts + warps) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_expert_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemMost);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_expert_sort, a);
  }
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
  return run_rows(fn, RowOp::kCombineBackward, a, dtype, stream);
}
