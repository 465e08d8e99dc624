// The block join: norms before and after a block fused with its gate and
// residual scale, and its gradient.  Argument checks, kernels, launches.
//
//   u = N_post(b)   (b itself without a post norm)
//   o = x + s g u   (g: none, a channel vector, a number a row, or full)
//   n = N_pre(o)    (the norm before the next block)
//   N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * w + bias, no mean and
//   no bias for rms.
//
// Backward, with t = dn w_pre, oh and bh the normalised rows, R the row's
// 1/deviation:
//   do' = do + R_o (t - mean(t) - oh mean(t oh))       (mean(t): layer only)
//   dx = do';  dg = sum over what g was spread over of s u do';  q = s g do' w_post
//   db = R_b (q - mean(q) - bh mean(q bh))
//   dw_pre = sum dn oh, dbias_pre = sum dn, dw_post = sum s g do' bh,
//   dbias_post = sum s g do', over the rows.
// The backward pass forms o again from x and b, which a training step holds
// anyway, so o's own rounding enters no gradient.
//
// What bounds it: bytes (forward: x, b in, o, n out; backward: x, b, do, dn
// in, dx, db out).  The kernels here take rows above 8192 channels, and those
// below of which not one fits into shared memory; the others are in
// zero_join_rows.cuh.
#include <cuda_runtime.h>
#include <inttypes.h>
#include <math.h>

#include <algorithm>

#include "zero_capi_util.h"
#include "zero_join_rows.cuh"

namespace zero {

// one translation unit a pair of types (zero_join_*.cu)
extern template int launch_join_rows<float, float>(const JoinArgs&, bool, int*, cudaStream_t);
extern template int launch_join_rows<__half, __half>(const JoinArgs&, bool, int*, cudaStream_t);
extern template int launch_join_rows<__half, float>(const JoinArgs&, bool, int*, cudaStream_t);
extern template int launch_join_rows<__nv_bfloat16, __nv_bfloat16>(const JoinArgs&, bool, int*, cudaStream_t);
extern template int launch_join_rows<__nv_bfloat16, float>(const JoinArgs&, bool, int*, cudaStream_t);

namespace {

// ---------------------------------------------------------------------------
// Rows of any length and alignment: a CTA a row, element by element, the row
// read again for each phase (from L1 or L2) and o formed again from it; the
// backward column sums are kept in the CTA's partials.  Bound by that work, not
// by bytes: 4096 x 12288 bf16, rms norms on both sides, 457 us forward and 2165
// backward (0.13 and 0.04 of a plain copy's bandwidth).

constexpr int kAnyThreads = 256;
constexpr int kAnyWorkers = 4 * kSMs;

// Sums of up to three values over the CTA, the same in every thread, in a
// fixed order.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* part) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_all_sum(v[k]);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[warp * N + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float t = part[k];
    for (int w = 1; w < warps; ++w) t += part[w * N + k];
    v[k] = t;
  }
  __syncthreads();
}

// One row's operands, by element.
template <class A, class R>
struct Row {
  const JoinArgs& a;
  const R* x;
  const A* b;
  int64_t row;
  float g_row;        // scale times the row's gate (row gates)
  float mb, rb, mo, ro;

  __device__ __forceinline__ Row(const JoinArgs& a_, int64_t r) : a(a_), row(r) {
    x = static_cast<const R*>(a.in.x) + r * a.d.x_stride;
    b = static_cast<const A*>(a.in.b) + (a.in.b ? r * a.d.b_stride : 0);
    g_row = a.scale;
    if (a.d.gate_kind == ZERO_GATE_ROW)
      g_row *= load_any(a.in.gate, r * a.d.gate_stride, a.d.gate_dtype);
    mb = mo = 0.f;
    rb = ro = 1.f;
  }
  __device__ __forceinline__ float gate(int64_t c) const {
    if (a.d.gate_kind == ZERO_GATE_CHANNEL) return a.scale * load_any(a.in.gate, c, a.d.gate_dtype);
    if (a.d.gate_kind == ZERO_GATE_FULL)
      return a.scale * load_any(a.in.gate, row * a.d.gate_stride + c, a.d.gate_dtype);
    return g_row;
  }
  // the row's or the element's own gate, without the scale
  __device__ __forceinline__ float own_gate(int64_t c) const {
    return load_any(a.in.gate, row * a.d.gate_stride + (a.d.gate_kind == ZERO_GATE_FULL ? c : 0), a.d.gate_dtype);
  }
  __device__ __forceinline__ float block(int64_t c) const { return Elem<A>::widen(b[c]); }
  __device__ __forceinline__ float b_hat(int64_t c) const { return (block(c) - mb) * rb; }
  __device__ __forceinline__ float u(int64_t c) const {
    if (!a.in.w_post) return block(c);
    float v = b_hat(c) * load_any(a.in.w_post, c, a.d.param_dtype);
    if (a.in.bias_post) v += load_any(a.in.bias_post, c, a.d.param_dtype);
    return v;
  }
  __device__ __forceinline__ float out(int64_t c) const {
    const float v = Elem<R>::widen(x[c]);
    return a.in.b ? fmaf(gate(c), u(c), v) : v;
  }
  __device__ __forceinline__ float o_hat(int64_t c) const { return (out(c) - mo) * ro; }
};

// Mean (layer only) and 1/deviation of value(c) over a row, two passes.
template <class F>
__device__ __forceinline__ void row_stats(const JoinArgs& a, F value, float* part, float& mean, float& r) {
  mean = 0.f;
  if (a.layer) {
    float s[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.d.hidden; c += blockDim.x) s[0] += value(c);
    block_sums(s, part);
    mean = s[0] * a.inv_h;
  }
  float s[1] = {0.f};
  for (int64_t c = threadIdx.x; c < a.d.hidden; c += blockDim.x) {
    const float v = value(c) - mean;
    s[0] = fmaf(v, v, s[0]);
  }
  block_sums(s, part);
  r = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
}

template <class A, class R>
__global__ void __launch_bounds__(kAnyThreads) k_join_any(const __grid_constant__ JoinArgs a) {
  __shared__ float part[kAnyThreads / 32];
  for (int64_t r = blockIdx.x; r < a.d.rows; r += gridDim.x) {
    Row<A, R> row(a, r);
    if (a.in.w_post) row_stats(a, [&](int64_t c) { return row.block(c); }, part, row.mb, row.rb);
    if (a.in.w_pre) row_stats(a, [&](int64_t c) { return row.out(c); }, part, row.mo, row.ro);
    if (a.stats && threadIdx.x == 0) a.stats[r] = make_float4(row.mb, row.rb, row.mo, row.ro);
    // the row's last reads come before its writes, element by element, so o
    // may be x and n may be b
    for (int64_t c = threadIdx.x; c < a.d.hidden; c += blockDim.x) {
      const float o = row.out(c);
      if (a.n) {
        float v = (o - row.mo) * row.ro * load_any(a.in.w_pre, c, a.d.param_dtype);
        if (a.in.bias_pre) v += load_any(a.in.bias_pre, c, a.d.param_dtype);
        static_cast<A*>(a.n)[r * a.d.hidden + c] = Elem<A>::narrow(v);
      }
      if (a.o) static_cast<R*>(a.o)[r * a.d.hidden + c] = Elem<R>::narrow(o);
    }
  }
}

template <class A, class R>
__global__ void __launch_bounds__(kAnyThreads) k_join_backward_any(const __grid_constant__ JoinArgs a) {
  __shared__ float part[3 * kAnyThreads / 32];
  const int64_t H = a.d.hidden;
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * a.n_sums * H;
  const bool by_row = a.d.gate_kind == ZERO_GATE_ROW || a.d.gate_kind == ZERO_GATE_FULL;
  for (int64_t r = blockIdx.x; r < a.d.rows; r += gridDim.x) {
    const bool first = r == blockIdx.x;
    Row<A, R> row(a, r);
    const float4 st = a.stats ? a.stats[r] : make_float4(0.f, 1.f, 0.f, 1.f);
    row.mb = st.x, row.rb = st.y, row.mo = st.z, row.ro = st.w;
    const R* d_o = a.d_o ? static_cast<const R*>(a.d_o) + r * a.d.do_stride : nullptr;
    const A* d_n = a.d_n ? static_cast<const A*>(a.d_n) + r * a.d.dn_stride : nullptr;
    float pre[2] = {0.f, 0.f};
    if (d_n) {
      for (int64_t c = threadIdx.x; c < H; c += blockDim.x) {
        const float t = Elem<A>::widen(d_n[c]) * load_any(a.in.w_pre, c, a.d.param_dtype);
        pre[0] += t;
        pre[1] = fmaf(t, row.o_hat(c), pre[1]);
      }
      block_sums(pre, part);
      pre[0] = a.layer ? pre[0] * a.inv_h : 0.f;
      pre[1] *= a.inv_h;
    }
    auto grad_o = [&](int64_t c) {
      float v = d_o ? Elem<R>::widen(d_o[c]) : 0.f;
      if (d_n) {
        const float t = Elem<A>::widen(d_n[c]) * load_any(a.in.w_pre, c, a.d.param_dtype);
        v = fmaf(row.ro, t - pre[0] - row.o_hat(c) * pre[1], v);
      }
      return v;
    };
    float post[3] = {0.f, 0.f, 0.f};
    const bool row_gate = a.d.gate_kind == ZERO_GATE_ROW && a.dgate;
    if ((a.in.w_post && a.db) || row_gate) {
      for (int64_t c = threadIdx.x; c < H; c += blockDim.x) {
        const float go = grad_o(c);
        if (a.in.w_post) {
          const float q = row.gate(c) * go * load_any(a.in.w_post, c, a.d.param_dtype);
          post[0] += q;
          post[1] = fmaf(q, row.b_hat(c), post[1]);
        }
        if (row_gate) post[2] = fmaf(a.scale * go, row.u(c), post[2]);
      }
      block_sums(post, part);
      post[0] = a.layer ? post[0] * a.inv_h : 0.f;
      post[1] *= a.inv_h;
      if (row_gate && threadIdx.x == 0) store_any(a.dgate, r, a.d.gate_dtype, post[2]);
    }
    for (int64_t c = threadIdx.x; c < H; c += blockDim.x) {
      const float go = grad_o(c);
      auto add = [&](int which, float v) {
        if (a.slot[which] < 0) return;
        float* p = mine + a.slot[which] * H + c;
        *p = first ? v : *p + v;
      };
      if (d_n) {
        const float dn = Elem<A>::widen(d_n[c]);
        add(kSumP, dn * row.o_hat(c));
        add(kSumQ, dn);
      }
      if (a.in.b) {
        const float du = row.gate(c) * go;
        const float y = by_row ? row.own_gate(c) * go : go;
        add(kSumS, y * (a.in.w_post ? row.b_hat(c) : row.block(c)));
        add(kSumB, y);
        if (a.d.gate_kind == ZERO_GATE_FULL && a.dgate)
          store_any(a.dgate, r * H + c, a.d.gate_dtype, a.scale * go * row.u(c));
        if (a.db) {
          float v = du;
          if (a.in.w_post)
            v = row.rb * (du * load_any(a.in.w_post, c, a.d.param_dtype) - post[0] - row.b_hat(c) * post[1]);
          static_cast<A*>(a.db)[r * H + c] = Elem<A>::narrow(v);
        }
      }
      if (a.dx) static_cast<R*>(a.dx)[r * H + c] = Elem<R>::narrow(go);
    }
  }
}

// Parameter gradients: a column's partials in kSumRows strands, each in
// worker order, then the strands in order.  A CTA has 16 columns, so that
// short rows make enough CTAs; a strand's loads of all sums are in flight
// together (with 8 strands of 32 columns this took 20 us for 760 workers).
constexpr int kSumRows = 64, kSumCols = 16, kSumAhead = 4;

__global__ void __launch_bounds__(kSumCols * kSumRows) k_join_sums(const __grid_constant__ JoinSumArgs g) {
  __shared__ float part[kJoinSums][kSumRows][kSumCols + 1];
  const JoinArgs& a = g.a;
  const int64_t H = a.d.hidden, c = static_cast<int64_t>(blockIdx.x) * kSumCols + threadIdx.x;
  float s[kJoinSums] = {0.f, 0.f, 0.f, 0.f};
  const float* p = a.partial + c;
  const int64_t worker = a.n_sums * H;
  wait_for_previous();
  if (c < H) {
    for (int w = threadIdx.y; w < g.workers; w += kSumAhead * kSumRows) {
      float v[kJoinSums][kSumAhead];
#pragma unroll
      for (int k = 0; k < kJoinSums; ++k)
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) {
          const int x = w + i * kSumRows;
          v[k][i] = a.slot[k] >= 0 && x < g.workers ? p[x * worker + a.slot[k] * H] : 0.f;
        }
#pragma unroll
      for (int k = 0; k < kJoinSums; ++k)
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) s[k] += v[k][i];
    }
  }
#pragma unroll
  for (int k = 0; k < kJoinSums; ++k) part[k][threadIdx.y][threadIdx.x] = s[k];
  __syncthreads();
  // strands 8 at a time, twice
  for (int rows = kSumRows / 8; rows > 0; rows /= 8) {
    float t[kJoinSums] = {0.f, 0.f, 0.f, 0.f};
    if (threadIdx.y < rows) {
#pragma unroll
      for (int k = 0; k < kJoinSums; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[k] += part[k][threadIdx.y * 8 + i][threadIdx.x];
    }
    __syncthreads();
    if (threadIdx.y < rows) {
#pragma unroll
      for (int k = 0; k < kJoinSums; ++k) part[k][threadIdx.y][threadIdx.x] = s[k] = t[k];
    }
    __syncthreads();
  }
  if (threadIdx.y != 0 || c >= H) return;
  const int pt = a.d.param_dtype;
  if (g.dw_pre) store_any(g.dw_pre, c, pt, s[kSumP]);
  if (g.dbias_pre) store_any(g.dbias_pre, c, pt, s[kSumQ]);
  float gate = a.scale;
  // (row and full gates are in the sums already)
  if (a.d.gate_kind == ZERO_GATE_CHANNEL) gate *= load_any(a.in.gate, c, a.d.gate_dtype);
  if (g.dw_post) store_any(g.dw_post, c, pt, gate * s[kSumS]);
  if (g.dbias_post) store_any(g.dbias_post, c, pt, gate * s[kSumB]);
  if (g.dgate) {
    float v = s[kSumS];
    if (a.in.w_post) v *= load_any(a.in.w_post, c, pt);
    if (a.in.bias_post) v = fmaf(load_any(a.in.bias_post, c, pt), s[kSumB], v);
    store_any(g.dgate, c, a.d.gate_dtype, a.scale * v);
  }
}

// CTAs that leave partials, at most.
int join_workers(const zero_join_desc& d) {
  int64_t most = kAnyWorkers;
  if (d.hidden <= kJoinRowMost) {
    const int threads = std::min(join_threads(d, true, true), join_threads(d, false, true));
    most = kSMs * std::max(1, kJoinThreadsBackward / threads);
  }
  return static_cast<int>(std::min(d.rows, most));
}

template <class A, class R>
int launch_any(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  void* args[] = {const_cast<JoinArgs*>(&a)};
  const void* fn = backward ? reinterpret_cast<const void*>(&k_join_backward_any<A, R>)
                            : reinterpret_cast<const void*>(&k_join_any<A, R>);
  const int grid = static_cast<int>(std::min<int64_t>(a.d.rows, backward ? join_workers(a.d) : 16 * kSMs));
  *workers = grid;
  return static_cast<int>(cudaLaunchKernel(fn, dim3(grid), dim3(kAnyThreads), args, 0, s));
}

template <class F>
int by_types(const zero_join_desc& d, F f) {
  if (d.act_dtype == ZERO_FP32) return f(float(), float());
  if (d.act_dtype == ZERO_BF16) {
    if (d.res_dtype == ZERO_FP32) return f(__nv_bfloat16(), float());
    return f(__nv_bfloat16(), __nv_bfloat16());
  }
  if (d.res_dtype == ZERO_FP32) return f(__half(), float());
  return f(__half(), __half());
}

}  // namespace

static int launch_join(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  return by_types(a.d, [&](auto act, auto res) {
    using A = decltype(act);
    using R = decltype(res);
    const int e = launch_join_rows<A, R>(a, backward, workers, s);
    return e == -1 ? launch_any<A, R>(a, backward, workers, s) : e;
  });
}

namespace {

// ---------------------------------------------------------------------------
// checks

zero_status check_desc(const char* fn, const zero_join_desc* d) {
  if (!d) return fail(ZERO_ERR_INVALID, "%s: desc is NULL", fn);
  if (d->rows < 0 || d->hidden < 1)
    return fail(ZERO_ERR_INVALID, "%s: need rows >= 0 and hidden >= 1", fn);
  if (d->hidden > INT32_MAX || d->rows > INT64_C(1) << 40)
    return fail(ZERO_ERR_INVALID, "%s: hidden is above 2^31-1 or rows above 2^40", fn);
  if (!known_type(d->act_dtype) || !known_type(d->res_dtype) || !known_type(d->param_dtype))
    return fail(ZERO_ERR_INVALID, "%s: unknown dtype", fn);
  if (d->res_dtype != d->act_dtype && d->res_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: res_dtype must be act_dtype or ZERO_FP32", fn);
  if (d->param_dtype != d->act_dtype && d->param_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: param_dtype must be act_dtype or ZERO_FP32", fn);
  if (d->kind != ZERO_JOIN_RMS && d->kind != ZERO_JOIN_LAYER)
    return fail(ZERO_ERR_INVALID, "%s: kind must be ZERO_JOIN_RMS or ZERO_JOIN_LAYER", fn);
  if (d->gate_kind < ZERO_GATE_NONE || d->gate_kind > ZERO_GATE_FULL)
    return fail(ZERO_ERR_INVALID, "%s: unknown gate_kind", fn);
  if (d->gate_kind != ZERO_GATE_NONE && d->gate_dtype != d->act_dtype && d->gate_dtype != ZERO_FP32)
    return fail(ZERO_ERR_INVALID, "%s: gate_dtype must be act_dtype or ZERO_FP32", fn);
  if (!(isfinite(d->eps) && d->eps > 0.0 && static_cast<float>(d->eps) > 0.f))
    return fail(ZERO_ERR_INVALID, "%s: eps must be finite and > 0 in binary32", fn);
  if (!isfinite(d->scale)) return fail(ZERO_ERR_INVALID, "%s: scale must be finite", fn);
  return ZERO_OK;
}

zero_status check_array(const char* fn, const char* what, const void* p, int type, bool needed) {
  if (!p) {
    if (needed) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, what);
    return ZERO_OK;
  }
  if (!aligned_to(p, type_bytes(type)))
    return fail(ZERO_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, what);
  return ZERO_OK;
}

zero_status check_stride(const char* fn, const char* what, const void* p, int64_t stride, int64_t least) {
  if (p && (stride < least || stride > INT64_C(1) << 40))
    return fail(ZERO_ERR_INVALID, "%s: %s_stride must be at least %" PRId64, fn, what, least);
  return ZERO_OK;
}

#define JOIN_TRY(x)                 \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)

zero_status check_inputs(const char* fn, const zero_join_desc& d, const zero_join_inputs* in, bool any_rows) {
  if (!in) return fail(ZERO_ERR_INVALID, "%s: inputs is NULL", fn);
  JOIN_TRY(check_array(fn, "x", in->x, d.res_dtype, any_rows));
  JOIN_TRY(check_array(fn, "b", in->b, d.act_dtype, false));
  JOIN_TRY(check_array(fn, "w_post", in->w_post, d.param_dtype, false));
  JOIN_TRY(check_array(fn, "bias_post", in->bias_post, d.param_dtype, false));
  JOIN_TRY(check_array(fn, "w_pre", in->w_pre, d.param_dtype, false));
  JOIN_TRY(check_array(fn, "bias_pre", in->bias_pre, d.param_dtype, false));
  JOIN_TRY(check_array(fn, "gate", in->gate, d.gate_dtype, d.gate_kind != ZERO_GATE_NONE && any_rows));
  if (d.gate_kind == ZERO_GATE_NONE && in->gate)
    return fail(ZERO_ERR_INVALID, "%s: gate given but gate_kind is ZERO_GATE_NONE", fn);
  if (!in->b && any_rows && (in->w_post || in->bias_post || d.gate_kind != ZERO_GATE_NONE))
    return fail(ZERO_ERR_INVALID, "%s: a post norm or a gate needs b", fn);
  if ((in->bias_post && !in->w_post) || (in->bias_pre && !in->w_pre))
    return fail(ZERO_ERR_INVALID, "%s: a bias needs its weight", fn);
  if (d.kind == ZERO_JOIN_RMS && (in->bias_post || in->bias_pre))
    return fail(ZERO_ERR_INVALID, "%s: ZERO_JOIN_RMS has no biases", fn);
  JOIN_TRY(check_stride(fn, "x", in->x, d.x_stride, d.hidden));
  JOIN_TRY(check_stride(fn, "b", in->b, d.b_stride, d.hidden));
  if (d.gate_kind == ZERO_GATE_FULL) JOIN_TRY(check_stride(fn, "gate", in->gate, d.gate_stride, d.hidden));
  if (d.gate_kind == ZERO_GATE_ROW) JOIN_TRY(check_stride(fn, "gate", in->gate, d.gate_stride, 1));
  return ZERO_OK;
}

Extent rows_extent(const char* name, const void* p, const zero_join_desc& d, int64_t stride, int type) {
  return {name, p, d.rows, stride * type_bytes(type), d.hidden * type_bytes(type)};
}
Extent vector_extent(const char* name, const void* p, const zero_join_desc& d, int type) {
  const int64_t bytes = d.hidden * type_bytes(type);
  return {name, p, 1, bytes, bytes};
}
Extent gate_extent(const void* p, const zero_join_desc& d) {
  if (d.gate_kind == ZERO_GATE_CHANNEL) return vector_extent("gate", p, d, d.gate_dtype);
  const int64_t pitch = d.gate_stride * type_bytes(d.gate_dtype);
  return {"gate", p, d.rows, pitch, (d.gate_kind == ZERO_GATE_FULL ? d.hidden : 1) * type_bytes(d.gate_dtype)};
}
zero_status pending(const char* fn) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(e));
  return ZERO_OK;
}

zero_status launched(const char* fn, int e) {
  if (e)
    return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(static_cast<cudaError_t>(e)));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return ZERO_OK;
}

JoinArgs base_args(const zero_join_desc& d, const zero_join_inputs& in) {
  JoinArgs a = {};
  a.d = d;
  a.in = in;
  a.layer = d.kind == ZERO_JOIN_LAYER;
  a.eps = static_cast<float>(d.eps);
  a.scale = static_cast<float>(d.scale);
  a.inv_h = 1.0f / static_cast<float>(d.hidden);
  for (int& s : a.slot) s = -1;
  return a;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_block_join(const zero_join_desc* desc, const zero_join_inputs* inputs, void* o,
                                       void* n, float* stats, void* stream) {
  const char* fn = "zero_block_join";
  clear_error();
  NvtxRange range(fn);
  JOIN_TRY(check_desc(fn, desc));
  const zero_join_desc& d = *desc;
  JOIN_TRY(check_inputs(fn, d, inputs, d.rows > 0));
  JOIN_TRY(check_array(fn, "o", o, d.res_dtype, false));
  JOIN_TRY(check_array(fn, "n", n, d.act_dtype, false));
  if (stats && !aligned_to(stats, 16)) return fail(ZERO_ERR_ALIGN, "%s: stats must be 16-byte aligned", fn);
  if (n && !inputs->w_pre) return fail(ZERO_ERR_INVALID, "%s: n needs w_pre", fn);
  if (d.rows == 0) return ZERO_OK;
  if (!o && !n) return fail(ZERO_ERR_INVALID, "%s: neither o nor n is wanted", fn);
  const zero_join_inputs& in = *inputs;
  const int64_t count = d.rows * d.hidden;
  JOIN_TRY(check_overlaps(fn,
                          {Extent::block("o", o, count * type_bytes(d.res_dtype), in.x),
                           Extent::block("n", n, count * type_bytes(d.act_dtype), in.b),
                           Extent::block("stats", stats, d.rows * 16)},
                          {rows_extent("x", in.x, d, d.x_stride, d.res_dtype),
                           rows_extent("b", in.b, d, d.b_stride, d.act_dtype), gate_extent(in.gate, d),
                           vector_extent("w_post", in.w_post, d, d.param_dtype),
                           vector_extent("bias_post", in.bias_post, d, d.param_dtype),
                           vector_extent("w_pre", in.w_pre, d, d.param_dtype),
                           vector_extent("bias_pre", in.bias_pre, d, d.param_dtype)}));
  JOIN_TRY(pending(fn));
  JoinArgs a = base_args(d, *inputs);
  a.o = o;
  a.n = n;
  a.stats = reinterpret_cast<float4*>(stats);
  if (!n && !stats) a.in.w_pre = nullptr;  // its statistics go nowhere
  int workers = 0;
  return launched(fn, launch_join(a, false, &workers, static_cast<cudaStream_t>(stream)));
}

extern "C" zero_status zero_block_join_workspace_bytes(const zero_join_desc* desc, int64_t* bytes) {
  const char* fn = "zero_block_join_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  JOIN_TRY(check_desc(fn, desc));
  *bytes = std::max<int64_t>(16, static_cast<int64_t>(join_workers(*desc)) * kJoinSums * desc->hidden * 4);
  return ZERO_OK;
}

extern "C" zero_status zero_block_join_backward(const zero_join_desc* desc, const zero_join_inputs* inputs,
                                                const void* d_o, const void* d_n, const float* stats,
                                                const zero_join_grads* grads, void* workspace,
                                                int64_t workspace_bytes, void* stream) {
  const char* fn = "zero_block_join_backward";
  clear_error();
  NvtxRange range(fn);
  JOIN_TRY(check_desc(fn, desc));
  const zero_join_desc& d = *desc;
  JOIN_TRY(check_inputs(fn, d, inputs, d.rows > 0));
  if (!grads) return fail(ZERO_ERR_INVALID, "%s: grads is NULL", fn);
  const zero_join_inputs& in = *inputs;
  const bool rows = d.rows > 0;
  JOIN_TRY(check_array(fn, "d_o", d_o, d.res_dtype, false));
  JOIN_TRY(check_array(fn, "d_n", d_n, d.act_dtype, false));
  JOIN_TRY(check_stride(fn, "do", d_o, d.do_stride, d.hidden));
  JOIN_TRY(check_stride(fn, "dn", d_n, d.dn_stride, d.hidden));
  if (rows && !d_o && !d_n) return fail(ZERO_ERR_INVALID, "%s: neither d_o nor d_n is given", fn);
  if (d_n && !in.w_pre) return fail(ZERO_ERR_INVALID, "%s: d_n needs w_pre", fn);
  if (rows && !stats && (in.w_post || d_n)) return fail(ZERO_ERR_INVALID, "%s: stats is NULL", fn);
  if (stats && !aligned_to(stats, 16)) return fail(ZERO_ERR_ALIGN, "%s: stats must be 16-byte aligned", fn);
  JOIN_TRY(check_array(fn, "dx", grads->dx, d.res_dtype, false));
  JOIN_TRY(check_array(fn, "db", grads->db, d.act_dtype, false));
  JOIN_TRY(check_array(fn, "dgate", grads->dgate, d.gate_dtype, false));
  if (rows && grads->db && !in.b) return fail(ZERO_ERR_INVALID, "%s: db needs b", fn);
  if (grads->dgate && d.gate_kind == ZERO_GATE_NONE)
    return fail(ZERO_ERR_INVALID, "%s: dgate given but gate_kind is ZERO_GATE_NONE", fn);
  JoinArgs a = base_args(d, in);
  a.d_o = d_o;
  a.d_n = d_n;
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
  a.dx = grads->dx;
  a.db = grads->db;
  const bool channel = d.gate_kind == ZERO_GATE_CHANNEL;
  struct Want {
    const char* name;
    void* out;
    const void* of;
    int type;
    bool pre, bias;
  };
  const Want wants[] = {{"dw_pre", grads->dw_pre, in.w_pre, d.param_dtype, true, false},
                        {"dbias_pre", grads->dbias_pre, in.w_pre, d.param_dtype, true, true},
                        {"dw_post", grads->dw_post, in.w_post, d.param_dtype, false, false},
                        {"dbias_post", grads->dbias_post, in.w_post, d.param_dtype, false, true}};
  for (const Want& w : wants) {
    if (!w.out) continue;
    JOIN_TRY(check_array(fn, w.name, w.out, w.type, false));
    if (rows && !w.of) return fail(ZERO_ERR_INVALID, "%s: %s needs its parameter", fn, w.name);
    if (d.kind == ZERO_JOIN_RMS && w.bias) return fail(ZERO_ERR_INVALID, "%s: ZERO_JOIN_RMS has no biases", fn);
    if (rows && !d_n && w.pre) return fail(ZERO_ERR_INVALID, "%s: %s needs d_n", fn, w.name);
  }
  void* const dgate = channel ? grads->dgate : nullptr;
  const bool wanted[kJoinSums] = {grads->dw_pre != nullptr, grads->dbias_pre != nullptr,
                                  grads->dw_post || dgate, grads->dbias_post || (dgate && in.bias_post)};
  for (int k = 0; k < kJoinSums; ++k)
    if (wanted[k]) a.slot[k] = a.n_sums++;
  if (d.gate_kind == ZERO_GATE_ROW || d.gate_kind == ZERO_GATE_FULL) a.dgate = grads->dgate;
  if (!a.dx && !a.db && !a.dgate && a.n_sums == 0)
    return rows ? fail(ZERO_ERR_INVALID, "%s: no gradient is wanted", fn) : ZERO_OK;
  if (a.n_sums > 0) {
    if (!workspace) return fail(ZERO_ERR_INVALID, "%s: workspace is NULL", fn);
    if (!aligned_to(workspace, 16)) return fail(ZERO_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    const int64_t need = static_cast<int64_t>(join_workers(d)) * a.n_sums * d.hidden * 4;
    if (workspace_bytes < need)
      return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn,
                  workspace_bytes, need);
    a.partial = static_cast<float*>(workspace);
  }
  const int64_t count = d.rows * d.hidden;
  const int64_t gates = channel ? d.hidden : d.gate_kind == ZERO_GATE_ROW ? d.rows : count;
  JOIN_TRY(check_overlaps(fn,
                          {Extent::block("dx", grads->dx, count * type_bytes(d.res_dtype), d_o),
                           Extent::block("db", grads->db, count * type_bytes(d.act_dtype), d_n),
                           Extent::block("dgate", grads->dgate, gates * type_bytes(d.gate_dtype)),
                           vector_extent("dw_post", grads->dw_post, d, d.param_dtype),
                           vector_extent("dbias_post", grads->dbias_post, d, d.param_dtype),
                           vector_extent("dw_pre", grads->dw_pre, d, d.param_dtype),
                           vector_extent("dbias_pre", grads->dbias_pre, d, d.param_dtype),
                           Extent::block("workspace", a.partial, join_workers(d) * a.n_sums * d.hidden * 4)},
                          {rows_extent("x", in.x, d, d.x_stride, d.res_dtype),
                           rows_extent("b", in.b, d, d.b_stride, d.act_dtype), gate_extent(in.gate, d),
                           vector_extent("w_post", in.w_post, d, d.param_dtype),
                           vector_extent("bias_post", in.bias_post, d, d.param_dtype),
                           vector_extent("w_pre", in.w_pre, d, d.param_dtype),
                           rows_extent("d_o", d_o, d, d.do_stride, d.res_dtype),
                           rows_extent("d_n", d_n, d, d.dn_stride, d.act_dtype),
                           Extent::block("stats", stats, d.rows * 16)}));
  JOIN_TRY(pending(fn));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int workers = 0;
  if (rows) JOIN_TRY(launched(fn, launch_join(a, true, &workers, s)));
  if (a.n_sums > 0) {
    if (!rows) {  // zeros, whatever the parameters and the gate hold (they may be NULL)
      a.in = {};
      a.d.gate_kind = ZERO_GATE_NONE;
      a.scale = 1.f;
    }
    JoinSumArgs g = {a, workers, grads->dw_pre, grads->dbias_pre, grads->dw_post, grads->dbias_post, dgate};
    void* args[] = {&g};
    const int e = static_cast<int>(
        launch_maybe_early(reinterpret_cast<const void*>(&k_join_sums),
                           dim3(static_cast<unsigned>((d.hidden + kSumCols - 1) / kSumCols)),
                           dim3(kSumCols, kSumRows), args, rows, s));
    JOIN_TRY(launched(fn, e));
  }
  return ZERO_OK;
}
