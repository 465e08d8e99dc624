// The block join for rows of at most 8192 channels: a row's values stay in
// registers, eight columns a thread, from the one read to the one write.
//
// Row split.  A CTA of ceil(hidden / 8) threads (whole warps) takes a row at a
// time, grid-stride; a row's sums go through one shuffle tree a warp and one
// barrier.  Small rows make small CTAs, several to an SM.
//
// Column maps.  kOct: thread t has columns 8t..8t+7, one 16-byte access of
// 16-bit data.  kQuad (a 32-bit array takes part): columns 4t..4t+3 and
// 4(T+t)..+3, so fp32 accesses are whole 512-byte runs a warp.  kAny: columns
// t + kT, element accesses, for odd row lengths and unaligned rows.
//
// Loads.  kOct and kQuad read ahead through a ring of rows in shared memory
// filled by asynchronous copies; every thread copies just the columns that it
// will use, so the ring needs no barrier, and waits for its own copies only.
// The parameters' vectors lie in shared memory the same way.  kAny reads its
// row directly and relies on other CTAs of the SM to overlap.
//
// Backward column sums are held in registers over all of a CTA's rows.  With
// go the gradient of o, v = bh (or b without a post norm) and y the gate where
// it varies by row (else 1), four sums give all parameter gradients:
//   P = sum dn oh, Q = sum dn, A = sum y go v, B = sum y go;
//   dw_pre = P, dbias_pre = Q, dw_post = s g A, dbias_post = s g B,
//   dgate = s (w_post A + bias_post B), or s A without a post norm,
// g being the channel gate (1 without one).
#pragma once

#include <algorithm>

#include "zero_join.cuh"

namespace zero {

constexpr int kJoinStagesMost = 4;
constexpr int kJoinSmemMost = 224 * 1024;  // of one SM's CTAs together
constexpr int kJoinScratch = 2 * 32 * 3 * 4 + 256;  // two buffers of the warps' sums

enum JoinMap { kOct, kQuad, kAny };

// What lies in the ring and in the vectors' part of shared memory; offsets in
// bytes, -1: absent.
struct JoinLayout {
  int32_t threads;
  int32_t stages, stage_bytes;
  int32_t x, b, d_o, d_n, gate;                 // within a stage
  int32_t w_post, bias_post, w_pre, bias_pre, gate_vec;  // from the vectors' start
  int32_t vec_bytes;
};

__device__ __forceinline__ uint32_t smem_of(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most `ahead` groups are in flight.
__device__ __forceinline__ void copies_wait(int ahead) {
  if (ahead == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (ahead == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (ahead == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

template <int MAP>
struct JoinCols {
  int t, T, hidden;
  __device__ __forceinline__ int col(int k) const {
    if constexpr (MAP == kOct) return 8 * t + k;
    if constexpr (MAP == kQuad) return k < 4 ? 4 * t + k : 4 * (T + t) + k - 4;
    return t + k * T;
  }
  __device__ __forceinline__ bool has(int k) const { return col(k) < hidden; }

  // This thread's part of a row (or vector) of elements of `type` into its
  // slots at shared-memory address `slot`.
  __device__ __forceinline__ void fetch(uint32_t slot, const void* row, int type) const {
    const char* p = static_cast<const char*>(row);
    if constexpr (MAP == kOct) {
      if (!has(0)) return;
      if (type == ZERO_FP32) {
        copy_async<16>(slot + 16 * t, p + 32 * t);
        copy_async<16>(slot + 16 * (T + t), p + 32 * t + 16);
      } else {
        copy_async<16>(slot + 16 * t, p + 16 * t);
      }
    } else if constexpr (MAP == kQuad) {
      if (type == ZERO_FP32) {
        if (has(0)) copy_async<16>(slot + 16 * t, p + 16 * t);
        if (has(4)) copy_async<16>(slot + 16 * (T + t), p + 16 * (T + t));
      } else {
        if (has(0)) copy_async<8>(slot + 8 * t, p + 8 * t);
        if (has(4)) copy_async<8>(slot + 8 * (T + t), p + 8 * (T + t));
      }
    }
  }
  // The same slots as binary32, zero past the row's end.
  __device__ __forceinline__ void read(const char* slot, int type, float (&v)[8]) const {
    if constexpr (MAP == kOct) {
      if (!has(0)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
      } else if (type == ZERO_FP32) {
        quad32(slot + 16 * t, v);
        quad32(slot + 16 * (T + t), v + 4);
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(slot + 16 * t);
        pair16(w.x, type, v), pair16(w.y, type, v + 2);
        pair16(w.z, type, v + 4), pair16(w.w, type, v + 6);
      }
    } else if constexpr (MAP == kQuad) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* q = v + 4 * h;
        if (!has(4 * h)) {
          q[0] = q[1] = q[2] = q[3] = 0.f;
        } else if (type == ZERO_FP32) {
          quad32(slot + 16 * (h * T + t), q);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(slot + 8 * (h * T + t));
          pair16(w.x, type, q), pair16(w.y, type, q + 2);
        }
      }
    } else {  // vectors only: binary32, one plane a column
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = reinterpret_cast<const float*>(slot)[k * T + t];
    }
  }
  // Straight from global memory (kAny, and full gates there).
  __device__ __forceinline__ void read_global(const void* row, int type, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = has(k) ? load_any(row, col(k), type) : 0.f;
  }
  template <class T_>
  __device__ __forceinline__ void write(T_* row, const float (&v)[8]) const {
    if constexpr (MAP == kOct) {
      if (has(0)) Elem<T_>::store8(row + 8 * t, v);
    } else if constexpr (MAP == kQuad) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (has(4 * h)) quad_out(row + 4 * (h * T + t), v + 4 * h);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (has(k)) row[col(k)] = Elem<T_>::narrow(v[k]);
    }
  }
  __device__ __forceinline__ void write_any(void* row, int64_t at, int type, const float (&v)[8]) const {
    if (type == ZERO_FP32)
      write(static_cast<float*>(row) + at, v);
    else if (type == ZERO_BF16)
      write(static_cast<__nv_bfloat16*>(row) + at, v);
    else
      write(static_cast<__half*>(row) + at, v);
  }

 private:
  static __device__ __forceinline__ void quad32(const char* p, float* v) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
  static __device__ __forceinline__ void pair16(uint32_t w, int type, float* v) {
    if (type == ZERO_BF16)
      Elem<__nv_bfloat16>::unpack(w, v[0], v[1]);
    else
      Elem<__half>::unpack(w, v[0], v[1]);
  }
  static __device__ __forceinline__ void quad_out(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  template <class T_>
  static __device__ __forceinline__ void quad_out(T_* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(Elem<T_>::pack(v[0], v[1]), Elem<T_>::pack(v[2], v[3]));
  }
};

// Sums of N values over the CTA, the same in every thread: a butterfly in the
// warp, one barrier, a butterfly over the warps' sums.  `flip` alternates
// between two buffers, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void join_sums(float (&v)[N], float* scratch, int& flip) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_all_sum(v[k]);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float* part = scratch + flip * 96;
  flip ^= 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k * 32 + warp] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_all_sum(lane < warps ? part[k * 32 + lane] : 0.f);
}

// The vectors (parameters, a channel gate) to this thread's slots.
template <int MAP>
__device__ __forceinline__ void fetch_vector(const JoinCols<MAP>& c, char* vec, int at, const void* p, int type) {
  if (at < 0) return;
  if constexpr (MAP == kAny) {
    float v[8];
    c.read_global(p, type, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) reinterpret_cast<float*>(vec + at)[k * c.T + c.t] = v[k];
  } else {
    c.fetch(smem_of(vec + at), p, type);
  }
}

template <int MAP>
__device__ __forceinline__ void read_vector(const JoinCols<MAP>& c, const char* vec, int at, int type, float (&v)[8]) {
  c.read(vec + at, MAP == kAny ? static_cast<int>(ZERO_FP32) : type, v);
}

// Row r's inputs into stage `stage`.
template <class A, class R, int MAP>
__device__ __forceinline__ void fetch_row(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP>& c,
                                          char* ring, int stage, int64_t r) {
  if constexpr (MAP != kAny) {
    if (r < a.d.rows) {
      const uint32_t s = smem_of(ring + stage * l.stage_bytes);
      c.fetch(s + l.x, static_cast<const R*>(a.in.x) + r * a.d.x_stride, Elem<R>::kType);
      if (l.b >= 0) c.fetch(s + l.b, static_cast<const A*>(a.in.b) + r * a.d.b_stride, Elem<A>::kType);
      if (l.d_o >= 0) c.fetch(s + l.d_o, static_cast<const R*>(a.d_o) + r * a.d.do_stride, Elem<R>::kType);
      if (l.d_n >= 0) c.fetch(s + l.d_n, static_cast<const A*>(a.d_n) + r * a.d.dn_stride, Elem<A>::kType);
      if (l.gate >= 0)
        c.fetch(s + l.gate,
                static_cast<const char*>(a.in.gate) + r * a.d.gate_stride * type_bytes(a.d.gate_dtype),
                a.d.gate_dtype);
    }
    copies_commit();
  }
}

// One input of row r: from the ring, or from global memory.
template <class E, int MAP>
__device__ __forceinline__ void row_input(const JoinCols<MAP>& c, const char* stage, int at, const void* p,
                                          int64_t r, int64_t stride, float (&v)[8]) {
  if constexpr (MAP == kAny) {
    const E* q = static_cast<const E*>(p) + r * stride;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c.has(k) ? Elem<E>::widen(q[c.col(k)]) : 0.f;
  } else {
    c.read(stage + at, Elem<E>::kType, v);
  }
}

// scale times the row's gate.
template <int MAP>
__device__ __forceinline__ void row_gate(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP>& c,
                                         const char* stage, const char* vec, int64_t r, float (&g)[8]) {
  if (a.d.gate_kind == ZERO_GATE_CHANNEL) {
    read_vector(c, vec, l.gate_vec, a.d.gate_dtype, g);
  } else if (a.d.gate_kind == ZERO_GATE_FULL) {
    if constexpr (MAP == kAny)
      c.read_global(static_cast<const char*>(a.in.gate) + r * a.d.gate_stride * type_bytes(a.d.gate_dtype),
                    a.d.gate_dtype, g);
    else
      c.read(stage + l.gate, a.d.gate_dtype, g);
  } else {
    const float one =
        a.d.gate_kind == ZERO_GATE_ROW ? load_any(a.in.gate, r * a.d.gate_stride, a.d.gate_dtype) : 1.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = one;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] *= a.scale;
}

// Mean (layer only) and 1/deviation of a row held by the CTA; v becomes the
// normalised row.
template <bool LAYER, int MAP>
__device__ __forceinline__ void normalise(const JoinArgs& a, const JoinCols<MAP>& c, float* scratch, int& flip,
                                          float (&v)[8], float& mean, float& r) {
  mean = 0.f;
  if constexpr (LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += c.has(k) ? v[k] : 0.f;
    join_sums(s, scratch, flip);
    mean = s[0] * a.inv_h;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = c.has(k) ? v[k] - mean : 0.f;
    s[0] = fmaf(v[k], v[k], s[0]);
  }
  join_sums(s, scratch, flip);
  r = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= r;
}

template <class A, class R, bool LAYER, int MAP, int MAXT>
__global__ void __launch_bounds__(MAXT, kJoinThreadsForward / MAXT) k_join_rows(const __grid_constant__ JoinArgs a,
                                                    const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  float* scratch = reinterpret_cast<float*>(smem);
  char* vec = smem + kJoinScratch;
  char* ring = vec + l.vec_bytes;
  const JoinCols<MAP> c = {static_cast<int>(threadIdx.x), l.threads, static_cast<int>(a.d.hidden)};
  int flip = 0;
  fetch_vector(c, vec, l.w_post, a.in.w_post, a.d.param_dtype);
  fetch_vector(c, vec, l.bias_post, a.in.bias_post, a.d.param_dtype);
  fetch_vector(c, vec, l.w_pre, a.in.w_pre, a.d.param_dtype);
  fetch_vector(c, vec, l.bias_pre, a.in.bias_pre, a.d.param_dtype);
  fetch_vector(c, vec, l.gate_vec, a.in.gate, a.d.gate_dtype);
  for (int s = 0; s < l.stages; ++s)
    fetch_row<A, R>(a, l, c, ring, s, blockIdx.x + static_cast<int64_t>(s) * gridDim.x);
  int stage = 0;
  for (int64_t r = blockIdx.x; r < a.d.rows; r += gridDim.x) {
    if constexpr (MAP != kAny) copies_wait(l.stages - 1);
    const char* in = ring + stage * l.stage_bytes;
    float o[8], v[8], mb = 0.f, rb = 1.f, mo = 0.f, ro = 1.f;
    row_input<R>(c, in, l.x, a.in.x, r, a.d.x_stride, o);
    if (a.in.b) {
      float g[8];
      row_input<A>(c, in, l.b, a.in.b, r, a.d.b_stride, v);
      row_gate(a, l, c, in, vec, r, g);
      if (a.in.w_post) {
        normalise<LAYER>(a, c, scratch, flip, v, mb, rb);
        float w[8];
        read_vector(c, vec, l.w_post, a.d.param_dtype, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= w[k];
        if (LAYER && a.in.bias_post) {
          read_vector(c, vec, l.bias_post, a.d.param_dtype, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += w[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(g[k], v[k], o[k]);
    }
    if (a.o) c.write(static_cast<R*>(a.o) + r * a.d.hidden, o);
    if (a.in.w_pre) {
      normalise<LAYER>(a, c, scratch, flip, o, mo, ro);
      if (a.n) {
        float w[8];
        read_vector(c, vec, l.w_pre, a.d.param_dtype, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] *= w[k];
        if (LAYER && a.in.bias_pre) {
          read_vector(c, vec, l.bias_pre, a.d.param_dtype, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] += w[k];
        }
        c.write(static_cast<A*>(a.n) + r * a.d.hidden, o);
      }
    }
    if (a.stats && threadIdx.x == 0) a.stats[r] = make_float4(mb, rb, mo, ro);
    // this thread has used its slots of the stage: the row `stages` ahead
    fetch_row<A, R>(a, l, c, ring, stage, r + static_cast<int64_t>(l.stages) * gridDim.x);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
  }
}

template <class A, class R, bool LAYER, int MAP, int MAXT>
__global__ void __launch_bounds__(MAXT) k_join_rows_backward(const __grid_constant__ JoinArgs a,
                                                             const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  float* scratch = reinterpret_cast<float*>(smem);
  char* vec = smem + kJoinScratch;
  char* ring = vec + l.vec_bytes;
  const JoinCols<MAP> c = {static_cast<int>(threadIdx.x), l.threads, static_cast<int>(a.d.hidden)};
  int flip = 0;
  fetch_vector(c, vec, l.w_post, a.in.w_post, a.d.param_dtype);
  fetch_vector(c, vec, l.bias_post, a.in.bias_post, a.d.param_dtype);
  fetch_vector(c, vec, l.w_pre, a.in.w_pre, a.d.param_dtype);
  fetch_vector(c, vec, l.gate_vec, a.in.gate, a.d.gate_dtype);
  for (int s = 0; s < l.stages; ++s)
    fetch_row<A, R>(a, l, c, ring, s, blockIdx.x + static_cast<int64_t>(s) * gridDim.x);
  const bool by_row = a.d.gate_kind == ZERO_GATE_ROW || a.d.gate_kind == ZERO_GATE_FULL;
  float P[8], Q[8], S[8], B[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) P[k] = Q[k] = S[k] = B[k] = 0.f;
  int stage = 0;
  for (int64_t r = blockIdx.x; r < a.d.rows; r += gridDim.x) {
    const float4 st = a.stats ? __ldg(a.stats + r) : make_float4(0.f, 1.f, 0.f, 1.f);
    if constexpr (MAP != kAny) copies_wait(l.stages - 1);
    const char* in = ring + stage * l.stage_bytes;
    float g[8], bh[8], go[8];
    if (a.d_o) {
      row_input<R>(c, in, l.d_o, a.d_o, r, a.d.do_stride, go);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) go[k] = 0.f;
    }
    if (a.in.b) {
      row_gate(a, l, c, in, vec, r, g);
      row_input<A>(c, in, l.b, a.in.b, r, a.d.b_stride, bh);
      if (a.in.w_post) {
#pragma unroll
        for (int k = 0; k < 8; ++k) bh[k] = (bh[k] - st.x) * st.y;
      }
    }
    if (a.d_n) {
      float oh[8], t[8], w[8];
      row_input<R>(c, in, l.x, a.in.x, r, a.d.x_stride, oh);
      if (a.in.b) {
        float u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = bh[k];
        if (a.in.w_post) {
          read_vector(c, vec, l.w_post, a.d.param_dtype, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] *= w[k];
          if (LAYER && a.in.bias_post) {
            read_vector(c, vec, l.bias_post, a.d.param_dtype, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] += w[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) oh[k] = fmaf(g[k], u[k], oh[k]);
      }
      row_input<A>(c, in, l.d_n, a.d_n, r, a.d.dn_stride, t);
      read_vector(c, vec, l.w_pre, a.d.param_dtype, w);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        oh[k] = (oh[k] - st.z) * st.w;
        P[k] = fmaf(t[k], oh[k], P[k]);
        if (LAYER) Q[k] += t[k];
        t[k] *= w[k];          // zero past the row's end, as dn is
        s[0] += t[k];
        s[1] = fmaf(t[k], oh[k], s[1]);
      }
      if constexpr (LAYER) {
        join_sums(s, scratch, flip);
        s[0] *= a.inv_h;
      } else {
        float one[1] = {s[1]};
        join_sums(one, scratch, flip);
        s[0] = 0.f, s[1] = one[0];
      }
      s[1] *= a.inv_h;
#pragma unroll
      for (int k = 0; k < 8; ++k) go[k] = fmaf(st.w, t[k] - s[0] - oh[k] * s[1], go[k]);
    }
    if (a.dx) c.write(static_cast<R*>(a.dx) + r * a.d.hidden, go);
    if (a.in.b) {
      const bool gate_row = a.d.gate_kind == ZERO_GATE_ROW && a.dgate;
      const bool gate_full = a.d.gate_kind == ZERO_GATE_FULL && a.dgate;
      float w[8], q[8], s[3] = {0.f, 0.f, 0.f};
      if (gate_row || gate_full) {
        float u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = bh[k];
        if (a.in.w_post) {
          read_vector(c, vec, l.w_post, a.d.param_dtype, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] *= w[k];
          if (LAYER && a.in.bias_post) {
            read_vector(c, vec, l.bias_post, a.d.param_dtype, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] += w[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          u[k] *= a.scale * go[k];
          s[2] += c.has(k) ? u[k] : 0.f;
        }
        if (gate_full) c.write_any(a.dgate, r * a.d.hidden, a.d.gate_dtype, u);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        q[k] = g[k] * go[k];                  // the gradient of u
        const float y = by_row ? q[k] : go[k];
        S[k] = fmaf(y, bh[k], S[k]);
        if (LAYER) B[k] += y;
      }
      if (a.in.w_post && (a.db || gate_row)) {
        read_vector(c, vec, l.w_post, a.d.param_dtype, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          q[k] = c.has(k) ? q[k] * w[k] : 0.f;
          s[0] += q[k];
          s[1] = fmaf(q[k], bh[k], s[1]);
        }
        join_sums(s, scratch, flip);
        s[0] = LAYER ? s[0] * a.inv_h : 0.f;
        s[1] *= a.inv_h;
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = st.y * (q[k] - s[0] - bh[k] * s[1]);
      } else if (gate_row) {
        float one[1] = {s[2]};
        join_sums(one, scratch, flip);
        s[2] = one[0];
      }
      if (gate_row && threadIdx.x == 0) store_any(a.dgate, r, a.d.gate_dtype, s[2]);
      if (a.db) c.write(static_cast<A*>(a.db) + r * a.d.hidden, q);
    }
    fetch_row<A, R>(a, l, c, ring, stage, r + static_cast<int64_t>(l.stages) * gridDim.x);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
  }
  if (a.n_sums == 0) return;
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * a.n_sums * a.d.hidden;
  auto leave = [&](int which, const float (&v)[8]) {
    if (a.slot[which] >= 0) c.write(mine + static_cast<int64_t>(a.slot[which]) * a.d.hidden, v);
  };
  leave(kSumP, P);
  leave(kSumS, S);
  if (LAYER) {
    leave(kSumQ, Q);
    leave(kSumB, B);
  }
}

// ---------------------------------------------------------------------------
// host: the layout and the launch of one type pair

inline int join_threads(int64_t hidden) { return static_cast<int>((hidden + 255) / 256 * 32); }

inline bool join_row_fits(const void* p, int64_t stride, int type, bool oct) {
  if (!p) return true;
  const int bytes = type_bytes(type);
  const int unit = oct || bytes == 4 ? 16 : 8;
  return aligned_to(p, unit) && stride * bytes % unit == 0;
}

// The column map these pointers and strides allow.
template <class A, class R>
JoinMap join_map(const JoinArgs& a) {
  const zero_join_desc& d = a.d;
  const bool oct = sizeof(A) == 2 && sizeof(R) == 2;
  if (d.hidden % (oct ? 8 : 4)) return kAny;
  const int64_t H = d.hidden;
  auto ok = [&](const void* p, int64_t stride, int type) { return join_row_fits(p, stride, type, oct); };
  const bool rows = ok(a.in.x, d.x_stride, d.res_dtype) && ok(a.in.b, d.b_stride, d.act_dtype) &&
                    ok(a.d_o, d.do_stride, d.res_dtype) && ok(a.d_n, d.dn_stride, d.act_dtype) &&
                    ok(a.o, H, d.res_dtype) && ok(a.n, H, d.act_dtype) && ok(a.dx, H, d.res_dtype) &&
                    ok(a.db, H, d.act_dtype);
  const bool full = d.gate_kind == ZERO_GATE_FULL;
  const bool gate = !full || (ok(a.in.gate, d.gate_stride, d.gate_dtype) && ok(a.dgate, H, d.gate_dtype));
  const void* vectors[] = {a.in.w_post, a.in.bias_post, a.in.w_pre, a.in.bias_pre,
                           d.gate_kind == ZERO_GATE_CHANNEL ? a.in.gate : nullptr};
  bool vec = true;
  for (const void* p : vectors) vec = vec && aligned_to(p, 16);
  if (!rows || !gate || !vec) return kAny;
  return oct ? kOct : kQuad;
}

inline JoinLayout join_layout(const JoinArgs& a, JoinMap map, bool backward, int ctas) {
  JoinLayout l = {};
  l.threads = join_threads(a.d.hidden);
  const int T8 = l.threads * 8;
  auto vector = [&](const void* p, int type) {
    if (!p) return -1;
    const int at = l.vec_bytes;
    l.vec_bytes += T8 * (map == kAny ? 4 : type_bytes(type));
    return at;
  };
  l.w_post = vector(a.in.w_post, a.d.param_dtype);
  l.bias_post = vector(a.in.bias_post, a.d.param_dtype);
  l.w_pre = vector(backward && !a.d_n ? nullptr : a.in.w_pre, a.d.param_dtype);
  l.bias_pre = vector(backward ? nullptr : a.in.bias_pre, a.d.param_dtype);
  l.gate_vec = vector(a.d.gate_kind == ZERO_GATE_CHANNEL ? a.in.gate : nullptr, a.d.gate_dtype);
  auto row = [&](const void* p, int type) {
    if (!p || map == kAny) return -1;
    const int at = l.stage_bytes;
    l.stage_bytes += T8 * type_bytes(type);
    return at;
  };
  l.x = row(a.in.x, a.d.res_dtype);
  l.b = row(a.in.b, a.d.act_dtype);
  l.d_o = row(a.d_o, a.d.res_dtype);
  l.d_n = row(a.d_n, a.d.act_dtype);
  l.gate = row(a.d.gate_kind == ZERO_GATE_FULL ? a.in.gate : nullptr, a.d.gate_dtype);
  if (map != kAny) {
    const int room = kJoinSmemMost / ctas - 1024 - kJoinScratch - l.vec_bytes;
    l.stages = std::max(0, std::min(kJoinStagesMost, room / l.stage_bytes));
  }
  return l;
}

inline int join_smem(const JoinLayout& l) { return kJoinScratch + l.vec_bytes + l.stages * l.stage_bytes; }

// CTAs of one SM: fewer of longer rows.
inline int join_ctas(int threads, bool backward) {
  return std::max(1, std::min(16, (backward ? kJoinThreadsBackward : kJoinThreadsForward) / threads));
}

template <class A, class R, bool LAYER, int MAP, int MAXT>
int launch_join_rows_as(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  const void* fn = backward ? reinterpret_cast<const void*>(&k_join_rows_backward<A, R, LAYER, MAP, MAXT>)
                            : reinterpret_cast<const void*>(&k_join_rows<A, R, LAYER, MAP, MAXT>);
  int ctas = join_ctas(join_threads(a.d.hidden), backward), fit = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, join_threads(a.d.hidden), 0);
  if (e != cudaSuccess) return static_cast<int>(e);
  ctas = std::max(1, std::min(ctas, fit));  // what the registers let run at once
  JoinLayout l = join_layout(a, static_cast<JoinMap>(MAP), backward, ctas);
  // two rows ahead before one more CTA
  while (ctas > 1 && ((MAP != kAny && l.stages < 2) || join_smem(l) > kJoinSmemMost / ctas - 1024)) {
    --ctas;
    l = join_layout(a, static_cast<JoinMap>(MAP), backward, ctas);
  }
  if (MAP != kAny && l.stages < 1) return -1;
  if (join_smem(l) > kJoinSmemMost) return -1;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmemMost);
  if (e != cudaSuccess) return static_cast<int>(e);
  const int grid = static_cast<int>(std::min<int64_t>(a.d.rows, static_cast<int64_t>(ctas) * kSMs));
  *workers = grid;
  JoinArgs copy = a;
  void* args[] = {&copy, &l};
  return static_cast<int>(cudaLaunchKernel(fn, dim3(grid), dim3(l.threads), args, join_smem(l), s));
}

template <class A, class R, bool LAYER, int MAP>
int launch_join_rows_map(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  // up to 512 threads a CTA leave 128 registers a thread, 1024 leave 64
  if (join_threads(a.d.hidden) <= 512) return launch_join_rows_as<A, R, LAYER, MAP, 512>(a, backward, workers, s);
  return launch_join_rows_as<A, R, LAYER, MAP, 1024>(a, backward, workers, s);
}

template <class A, class R, bool LAYER>
int launch_join_rows_kind(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  constexpr int kWide = sizeof(A) == 2 && sizeof(R) == 2 ? kOct : kQuad;
  int e = -1;
  if (join_map<A, R>(a) != kAny) e = launch_join_rows_map<A, R, LAYER, kWide>(a, backward, workers, s);
  if (e == -1) e = launch_join_rows_map<A, R, LAYER, kAny>(a, backward, workers, s);
  return e;
}

// -1: these rows do not fit here.
template <class A, class R>
int launch_join_rows(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  if (a.d.hidden > kJoinRowMost) return -1;
  return a.layer ? launch_join_rows_kind<A, R, true>(a, backward, workers, s)
                 : launch_join_rows_kind<A, R, false>(a, backward, workers, s);
}

}  // namespace zero
