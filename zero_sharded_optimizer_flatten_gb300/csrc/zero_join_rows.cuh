// The block join for rows of at most 8192 channels: a row's values stay in
// registers, eight columns a thread, from the one read to the one write.
//
// Row split.  Above 256 channels a CTA of ceil(hidden / 8) threads (whole
// warps) takes a row at a time; a row's sums go through one shuffle tree a
// warp and one barrier.  Up to 256 channels 8, 16 or 32 lanes take a row and
// a CTA of 128 threads several rows, without barriers.  Rows are handed out
// grid-stride.
//
// Column maps.  kOct: thread t of a row's T has columns 8t..8t+7, one 16-byte
// access of 16-bit data.  kQuad (a 32-bit array takes part): columns 4t..4t+3
// and 4(T+t)..+3, so fp32 accesses are whole 512-byte runs a warp.  kAny:
// columns t + kT, element accesses, for odd row lengths and unaligned rows.
//
// Loads.  kOct and kQuad read ahead through a ring of rows in shared memory
// filled by asynchronous copies; every thread copies just the columns that it
// will use, so the ring needs no barrier, and waits for its own copies only.
// kAny reads its row directly and relies on other CTAs of the SM to overlap.
//
// Arithmetic is in pairs of binary32 (two elements an instruction): with the
// loads asynchronous, the instructions issued a row are what stands beside
// the bytes.  What is the same for every row is folded beforehand into
// binary32 vectors in shared memory, zero past the row's end:
//   w1 = scale * (channel gate) * w_post, b1 = scale * (channel gate) *
//   bias_post, w2 = w_pre, b2 = bias_pre, so that o = x + y (w1 bh + b1), y
//   being a row's or an element's own gate or 1.
//
// Backward column sums are held in registers over all of a CTA's rows.  With
// go the gradient of o and v = bh (or b without a post norm), four sums give
// all parameter gradients:
//   P = sum dn oh, Q = sum dn, S = sum y go v, B = sum y go;
//   dw_pre = P, dbias_pre = Q, dw_post = s g S, dbias_post = s g B,
//   dgate = s (w_post S + bias_post B), or s S without a post norm,
// g being the channel gate (1 without one).
#pragma once

#include <algorithm>

#include "zero_join.cuh"

namespace zero {

constexpr int kJoinStagesMost = 4;
constexpr int kJoinSmemMost = 224 * 1024;  // of one SM's CTAs together
constexpr int kJoinScratch = 2 * 2 * 32 * 4;  // two buffers of two sums a warp
constexpr int kJoinSmallCta = 128;         // threads of a CTA of several rows

enum JoinMap { kOct, kQuad, kAny };

// What lies in the ring and in the vectors' part of shared memory; offsets in
// bytes, -1: absent.
struct JoinLayout {
  int32_t lanes;                    // threads of a row
  int32_t stages, stage_bytes;
  int32_t x, b, d_o, d_n, gate;     // within a stage
  int32_t w1, b1, w2, b2;           // from the vectors' start
  int32_t vec_bytes;
};

// Two binary32 values that go through one instruction.
struct F2 {
  uint64_t w;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.w) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ void f2_out(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.w));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.w) : "l"(a.w), "l"(b.w), "l"(c.w));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  float lo, hi;
  f2_out(a, lo, hi);
  return lo + hi;
}

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

template <class T>
__device__ __forceinline__ F2 widen2(uint32_t w) {
  float lo, hi;
  Elem<T>::unpack(w, lo, hi);
  return f2(lo, hi);
}
__device__ __forceinline__ F2 widen2_any(uint32_t w, int type) {
  return type == ZERO_BF16 ? widen2<__nv_bfloat16>(w) : widen2<__half>(w);
}
template <class T>
__device__ __forceinline__ uint32_t pack2(F2 v) {
  float lo, hi;
  f2_out(v, lo, hi);
  return Elem<T>::pack(lo, hi);
}

// A thread's eight columns of a row; in registers they are four pairs.
template <int MAP>
struct JoinCols {
  int t, T;        // place among the row's threads
  int tid, n;      // place in the CTA: where its slots are
  int hidden;
  __device__ __forceinline__ int col(int k) const {
    if constexpr (MAP == kOct) return 8 * t + k;
    if constexpr (MAP == kQuad) return k < 4 ? 4 * t + k : 4 * (T + t) + k - 4;
    return t + k * T;
  }
  __device__ __forceinline__ bool has(int k) const { return col(k) < hidden; }
  __device__ __forceinline__ bool ragged() const { return !has(7); }

  // This thread's part of a row of elements of `type` into its slots at
  // shared-memory address `slot`.
  __device__ __forceinline__ void fetch(uint32_t slot, const void* row, int type) const {
    const char* p = static_cast<const char*>(row);
    if constexpr (MAP == kOct) {
      if (!has(0)) return;
      if (type == ZERO_FP32) {
        copy_async<16>(slot + 16 * tid, p + 32 * t);
        copy_async<16>(slot + 16 * (n + tid), p + 32 * t + 16);
      } else {
        copy_async<16>(slot + 16 * tid, p + 16 * t);
      }
    } else if constexpr (MAP == kQuad) {
      if (type == ZERO_FP32) {
        if (has(0)) copy_async<16>(slot + 16 * tid, p + 16 * t);
        if (has(4)) copy_async<16>(slot + 16 * (n + tid), p + 16 * (T + t));
      } else {
        if (has(0)) copy_async<8>(slot + 8 * tid, p + 8 * t);
        if (has(4)) copy_async<8>(slot + 8 * (n + tid), p + 8 * (T + t));
      }
    }
  }
  // The same slots (cleared once where there is no column).
  template <class E>
  __device__ __forceinline__ void read(const char* slot, F2 (&v)[4]) const {
    if constexpr (Elem<E>::kType == ZERO_FP32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) quad32(slot + 16 * (h * n + tid), v + 2 * h);
    } else if constexpr (MAP == kOct) {
      const uint4 w = *reinterpret_cast<const uint4*>(slot + 16 * tid);
      v[0] = widen2<E>(w.x), v[1] = widen2<E>(w.y), v[2] = widen2<E>(w.z), v[3] = widen2<E>(w.w);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 w = *reinterpret_cast<const uint2*>(slot + 8 * (h * n + tid));
        v[2 * h] = widen2<E>(w.x), v[2 * h + 1] = widen2<E>(w.y);
      }
    }
  }
  __device__ __forceinline__ void read_any(const char* slot, int type, F2 (&v)[4]) const {
    if (type == ZERO_FP32)
      read<float>(slot, v);
    else if (type == ZERO_BF16)
      read<__nv_bfloat16>(slot, v);
    else
      read<__half>(slot, v);
  }
  // Straight from global memory, element by element.
  template <class E>
  __device__ __forceinline__ void read_global(const E* row, F2 (&v)[4]) const {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = has(k) ? Elem<E>::widen(row[col(k)]) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = f2(f[2 * k], f[2 * k + 1]);
  }
  __device__ __forceinline__ void read_global_any(const void* row, int64_t at, int type, F2 (&v)[4]) const {
    if (type == ZERO_FP32)
      read_global(static_cast<const float*>(row) + at, v);
    else if (type == ZERO_BF16)
      read_global(static_cast<const __nv_bfloat16*>(row) + at, v);
    else
      read_global(static_cast<const __half*>(row) + at, v);
  }
  // A vector's slots: this thread's eight binary32 values, two planes.
  __device__ __forceinline__ void vector_in(char* vec, const float (&f)[8]) const {
    *reinterpret_cast<float4*>(vec + 16 * tid) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(vec + 16 * (n + tid)) = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void vector(const char* vec, F2 (&v)[4]) const {
    quad32(vec + 16 * tid, v);
    quad32(vec + 16 * (n + tid), v + 2);
  }
  template <class E>
  __device__ __forceinline__ void write(E* row, const F2 (&v)[4]) const {
    if constexpr (MAP == kAny) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f2_out(v[k], lo, hi);
        if (has(2 * k)) row[col(2 * k)] = Elem<E>::narrow(lo);
        if (has(2 * k + 1)) row[col(2 * k + 1)] = Elem<E>::narrow(hi);
      }
    } else if constexpr (Elem<E>::kType == ZERO_FP32) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (has(4 * h))
          *reinterpret_cast<ulonglong2*>(row + col(4 * h)) = make_ulonglong2(v[2 * h].w, v[2 * h + 1].w);
    } else if constexpr (MAP == kOct) {
      if (has(0))
        *reinterpret_cast<uint4*>(row + col(0)) =
            make_uint4(pack2<E>(v[0]), pack2<E>(v[1]), pack2<E>(v[2]), pack2<E>(v[3]));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (has(4 * h))
          *reinterpret_cast<uint2*>(row + col(4 * h)) = make_uint2(pack2<E>(v[2 * h]), pack2<E>(v[2 * h + 1]));
    }
  }
  __device__ __forceinline__ void write_any(void* row, int64_t at, int type, const F2 (&v)[4]) const {
    if (type == ZERO_FP32)
      write(static_cast<float*>(row) + at, v);
    else if (type == ZERO_BF16)
      write(static_cast<__nv_bfloat16*>(row) + at, v);
    else
      write(static_cast<__half*>(row) + at, v);
  }

 private:
  static __device__ __forceinline__ void quad32(const char* p, F2* v) {
    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(p);
    v[0].w = f.x, v[1].w = f.y;
  }
};

// Sums of N <= 2 values over a row's threads, the same in all of them, in a
// fixed order: a butterfly over the row's lanes of a warp, then (rows of
// several warps) one barrier and the warps' sums in one order.  `flip`
// alternates between two buffers, so one barrier a sum is enough; sums of
// warps that the CTA lacks stay zero.
template <int QUADS, int N>
__device__ __forceinline__ void join_sums(float (&v)[N], float* scratch, int& flip, int lanes) {
  if constexpr (QUADS == 1) {  // rows of a warp or less
#pragma unroll
    for (int k = 0; k < N; ++k)
      for (int o = lanes >> 1; o > 0; o >>= 1) v[k] += __shfl_xor_sync(kFull, v[k], o);
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_all_sum(v[k]);
  float* part = scratch + flip * 64;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k * 32 + (threadIdx.x >> 5)] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(part + k * 32);
    F2 s[2];
    s[0].w = p[0].x, s[1].w = p[0].y;
#pragma unroll
    for (int w = 1; w < QUADS; ++w) {
      F2 q[2];
      q[0].w = p[w].x, q[1].w = p[w].y;
      s[0] = add2(s[0], q[0]);
      s[1] = add2(s[1], q[1]);
    }
    v[k] = sum2(add2(s[0], s[1]));
  }
}

// w1, b1, w2, b2 (see above) to this thread's slots.
template <int MAP>
__device__ __forceinline__ void fold_vectors(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP>& c,
                                             char* vec) {
  float f[8];
  auto each = [&](int at, auto value) {
    if (at < 0) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = c.has(k) ? value(c.col(k)) : 0.f;
    c.vector_in(vec + at, f);
  };
  const int pt = a.d.param_dtype;
  auto gate = [&](int k) {
    return a.d.gate_kind == ZERO_GATE_CHANNEL ? a.scale * load_any(a.in.gate, k, a.d.gate_dtype) : a.scale;
  };
  each(l.w1, [&](int k) { return a.in.w_post ? gate(k) * load_any(a.in.w_post, k, pt) : gate(k); });
  each(l.b1, [&](int k) { return gate(k) * load_any(a.in.bias_post, k, pt); });
  each(l.w2, [&](int k) { return load_any(a.in.w_pre, k, pt); });
  each(l.b2, [&](int k) { return load_any(a.in.bias_pre, k, pt); });
}

// Row r's inputs into stage `stage`.
template <class A, class R, int MAP>
__device__ __forceinline__ void fetch_row(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP>& c,
                                          char* ring, int stage, int64_t r) {
  if constexpr (MAP != kAny) {
    if (r < a.d.rows) {
      const uint32_t s = smem_of(ring) + stage * l.stage_bytes;
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
                                          int64_t r, int64_t stride, F2 (&v)[4]) {
  if constexpr (MAP == kAny)
    c.read_global(static_cast<const E*>(p) + r * stride, v);
  else
    c.template read<E>(stage + at, v);
}

// y w1: what multiplies the normalised block output, and y itself where rows
// or elements have their own gates (OWN).
template <bool OWN, int MAP>
__device__ __forceinline__ void row_gate(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP>& c,
                                         const char* stage, const char* vec, int64_t r, F2 (&y)[4],
                                         F2 (&w)[4]) {
  c.vector(vec + l.w1, w);
  if constexpr (OWN) {
    if (a.d.gate_kind == ZERO_GATE_FULL) {
      if constexpr (MAP == kAny)
        c.read_global_any(a.in.gate, r * a.d.gate_stride, a.d.gate_dtype, y);
      else
        c.read_any(stage + l.gate, a.d.gate_dtype, y);
    } else {
      y[0] = y[1] = y[2] = y[3] = f2(load_any(a.in.gate, r * a.d.gate_stride, a.d.gate_dtype));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = mul2(w[k], y[k]);
  }
}

// Mean (layer only) and 1/deviation of a row; v becomes the normalised row.
template <bool LAYER, int QUADS, int MAP>
__device__ __forceinline__ void normalise(const JoinArgs& a, const JoinCols<MAP>& c, float* scratch, int& flip,
                                          F2 (&v)[4], float& mean, float& r) {
  mean = 0.f;
  if constexpr (LAYER) {
    float s[1] = {sum2(add2(add2(v[0], v[1]), add2(v[2], v[3])))};
    join_sums<QUADS>(s, scratch, flip, c.T);
    mean = s[0] * a.inv_h;
    const F2 m = f2(-mean);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = add2(v[k], m);
    if (c.ragged()) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f2_out(v[k], lo, hi);
        v[k] = f2(c.has(2 * k) ? lo : 0.f, c.has(2 * k + 1) ? hi : 0.f);
      }
    }
  }
  F2 q = mul2(v[0], v[0]), p = mul2(v[1], v[1]);
  q = fma2(v[2], v[2], q), p = fma2(v[3], v[3], p);
  float s[1] = {sum2(add2(q, p))};
  join_sums<QUADS>(s, scratch, flip, c.T);
  r = rsqrtf(fmaf(s[0], a.inv_h, a.eps));
  const F2 rr = f2(r);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], rr);
}

// What both kernels set up.
template <int MAP, bool MANY>
struct JoinCta {
  float* scratch;
  char *vec, *ring;
  JoinCols<MAP> c;
  int64_t first, step;  // rows: first + i * step, while the CTA has any
  int group;            // this thread's row among the CTA's
  __device__ __forceinline__ JoinCta(const JoinArgs& a, const JoinLayout& l, char* smem) {
    scratch = reinterpret_cast<float*>(smem);
    vec = smem + kJoinScratch;
    ring = vec + l.vec_bytes;
    const int tid = static_cast<int>(threadIdx.x), n = static_cast<int>(blockDim.x);
    const int groups = MANY ? n / l.lanes : 1;
    group = MANY ? tid / l.lanes : 0;
    c.t = MANY ? tid % l.lanes : tid, c.T = MANY ? l.lanes : n, c.tid = tid, c.n = n, c.hidden = static_cast<int>(a.d.hidden);
    first = static_cast<int64_t>(blockIdx.x) * groups;
    step = static_cast<int64_t>(gridDim.x) * groups;
    // sums of warps the CTA lacks, and slots of columns a row lacks
    for (int i = tid; i < kJoinScratch / 4; i += n) scratch[i] = 0.f;
    for (int i = tid; i < l.stages * l.stage_bytes / 16; i += n)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
};

template <class A, class R, bool LAYER, bool OWN, int MAP, int MAXT>
__global__ void __launch_bounds__(MAXT, kJoinThreadsForward / MAXT) k_join_rows(
    const __grid_constant__ JoinArgs a, const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  constexpr bool kMany = MAXT == kJoinSmallCta;  // several rows a CTA
  constexpr int kQuads = MAXT / 128;              // a row's warps in fours
  JoinCta<MAP, kMany> cta(a, l, smem);
  const JoinCols<MAP>& c = cta.c;
  int flip = 0, stage = 0;
  for (int s = 0; s < l.stages; ++s)
    fetch_row<A, R>(a, l, c, cta.ring, s, cta.first + cta.group + s * cta.step);
  fold_vectors(a, l, c, cta.vec);
  for (int64_t base = cta.first; base < a.d.rows; base += cta.step) {
    // a group past the last row works on it once more and writes nothing
    const int64_t r = kMany ? min(base + cta.group, a.d.rows - 1) : base;
    const bool live = !kMany || base + cta.group < a.d.rows;
    if constexpr (MAP != kAny) copies_wait(l.stages - 1);
    const char* in = cta.ring + stage * l.stage_bytes;
    F2 o[4];
    float mb = 0.f, rb = 1.f, mo = 0.f, ro = 1.f;
    row_input<R>(c, in, l.x, a.in.x, r, a.d.x_stride, o);
    if (a.in.b) {
      F2 v[4], y[4], w[4];
      row_input<A>(c, in, l.b, a.in.b, r, a.d.b_stride, v);
      if (a.in.w_post) normalise<LAYER, kQuads>(a, c, cta.scratch, flip, v, mb, rb);
      row_gate<OWN>(a, l, c, in, cta.vec, r, y, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fma2(w[k], v[k], o[k]);
      if (LAYER && l.b1 >= 0) {
        c.vector(cta.vec + l.b1, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = OWN ? fma2(w[k], y[k], o[k]) : add2(w[k], o[k]);
      }
    }
    // this thread has read its slots of the stage: the row `stages` ahead
    fetch_row<A, R>(a, l, c, cta.ring, stage, base + cta.group + l.stages * cta.step);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
    if (a.o && live) c.write(static_cast<R*>(a.o) + r * a.d.hidden, o);
    if (a.in.w_pre) {
      normalise<LAYER, kQuads>(a, c, cta.scratch, flip, o, mo, ro);
      if (a.n && live) {
        F2 w[4];
        c.vector(cta.vec + l.w2, w);
        if (LAYER && l.b2 >= 0) {
          F2 d[4];
          c.vector(cta.vec + l.b2, d);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = fma2(o[k], w[k], d[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = mul2(o[k], w[k]);
        }
        c.write(static_cast<A*>(a.n) + r * a.d.hidden, o);
      }
    }
    if (a.stats && live && c.t == 0) a.stats[r] = make_float4(mb, rb, mo, ro);
  }
}

template <class A, class R, bool LAYER, bool OWN, int MAP, int MAXT>
__global__ void __launch_bounds__(MAXT) k_join_rows_backward(const __grid_constant__ JoinArgs a,
                                                             const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  constexpr bool kMany = MAXT == kJoinSmallCta;  // several rows a CTA
  constexpr int kQuads = MAXT / 128;              // a row's warps in fours
  JoinCta<MAP, kMany> cta(a, l, smem);
  const JoinCols<MAP>& c = cta.c;
  int flip = 0, stage = 0;
  for (int s = 0; s < l.stages; ++s)
    fetch_row<A, R>(a, l, c, cta.ring, s, cta.first + cta.group + s * cta.step);
  fold_vectors(a, l, c, cta.vec);
  const bool gate_row = OWN && a.d.gate_kind == ZERO_GATE_ROW && a.dgate;
  const bool gate_full = OWN && a.d.gate_kind == ZERO_GATE_FULL && a.dgate;
  F2 P[4], Q[4], S[4], B[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) P[k] = Q[k] = S[k] = B[k] = f2(0.f);
  float4 st = make_float4(0.f, 1.f, 0.f, 1.f);
  if (a.stats && cta.first < a.d.rows) st = __ldg(a.stats + min(cta.first + cta.group, a.d.rows - 1));
  for (int64_t base = cta.first; base < a.d.rows; base += cta.step) {
    const int64_t r = kMany ? min(base + cta.group, a.d.rows - 1) : base;
    const bool live = !kMany || base + cta.group < a.d.rows;
    const float4 now = st;
    if (a.stats) st = __ldg(a.stats + min(r + cta.step, a.d.rows - 1));  // the next row's
    if constexpr (MAP != kAny) copies_wait(l.stages - 1);
    const char* in = cta.ring + stage * l.stage_bytes;
    F2 go[4], bh[4], y[4], w1[4];
    if (a.d_o) {
      row_input<R>(c, in, l.d_o, a.d_o, r, a.d.do_stride, go);
    } else {
      go[0] = go[1] = go[2] = go[3] = f2(0.f);
    }
    if (a.in.b) {
      row_gate<OWN>(a, l, c, in, cta.vec, r, y, w1);
      row_input<A>(c, in, l.b, a.in.b, r, a.d.b_stride, bh);
      if (a.in.w_post) {
        const F2 rr = f2(now.y), m = f2(-now.x);
#pragma unroll
        for (int k = 0; k < 4; ++k) bh[k] = mul2(LAYER ? add2(bh[k], m) : bh[k], rr);
      }
    }
    if (a.d_n) {
      F2 oh[4], t[4], w[4];
      row_input<R>(c, in, l.x, a.in.x, r, a.d.x_stride, oh);
      row_input<A>(c, in, l.d_n, a.d_n, r, a.d.dn_stride, t);
      if (a.in.b) {
#pragma unroll
        for (int k = 0; k < 4; ++k) oh[k] = fma2(w1[k], bh[k], oh[k]);
        if (LAYER && l.b1 >= 0) {
          c.vector(cta.vec + l.b1, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) oh[k] = OWN ? fma2(w[k], y[k], oh[k]) : add2(w[k], oh[k]);
        }
      }
      c.vector(cta.vec + l.w2, w);
      const F2 rr = f2(now.w), m = f2(-now.z);
      F2 s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        oh[k] = mul2(LAYER ? add2(oh[k], m) : oh[k], rr);
        if (live) {
          P[k] = fma2(t[k], oh[k], P[k]);
          if (LAYER) Q[k] = add2(Q[k], t[k]);
        }
        t[k] = mul2(t[k], w[k]);  // zero past the row's end, as dn and w2 are
        if (LAYER) s0 = add2(s0, t[k]);
        s1 = fma2(t[k], oh[k], s1);
      }
      if constexpr (LAYER) {
        float s[2] = {sum2(s1), sum2(s0)};
        join_sums<kQuads>(s, cta.scratch, flip, c.T);
        s1 = f2(-s[0] * a.inv_h), s0 = f2(-s[1] * a.inv_h);
      } else {
        float s[1] = {sum2(s1)};
        join_sums<kQuads>(s, cta.scratch, flip, c.T);
        s1 = f2(-s[0] * a.inv_h);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        F2 e = fma2(oh[k], s1, t[k]);
        if (LAYER) e = add2(e, s0);
        go[k] = fma2(e, rr, go[k]);
      }
    }
    fetch_row<A, R>(a, l, c, cta.ring, stage, base + cta.group + l.stages * cta.step);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
    if (a.dx && live) c.write(static_cast<R*>(a.dx) + r * a.d.hidden, go);
    if (!a.in.b) continue;
    if (live) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const F2 yg = OWN ? mul2(y[k], go[k]) : go[k];
        S[k] = fma2(yg, bh[k], S[k]);
        if (LAYER) B[k] = add2(B[k], yg);
      }
    }
    float s2 = 0.f;
    if (gate_row || gate_full) {
      F2 u[4], w[4], sum = f2(0.f);
      c.vector(cta.vec + l.w1, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = mul2(w[k], bh[k]);
      if (LAYER && l.b1 >= 0) {
        c.vector(cta.vec + l.b1, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = add2(u[k], w[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = mul2(u[k], go[k]);
        sum = add2(sum, u[k]);
      }
      s2 = sum2(sum);
      if (gate_full && live) c.write_any(a.dgate, r * a.d.hidden, a.d.gate_dtype, u);
    }
    if (gate_row) {
      float one[1] = {s2};
      join_sums<kQuads>(one, cta.scratch, flip, c.T);
      if (live && c.t == 0) store_any(a.dgate, r, a.d.gate_dtype, one[0]);
    }
    if (!a.db) continue;
    F2 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = mul2(w1[k], go[k]);  // zero past the row's end, as w1 is
    if (a.in.w_post) {
      F2 s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (LAYER) s0 = add2(s0, q[k]);
        s1 = fma2(q[k], bh[k], s1);
      }
      if constexpr (LAYER) {
        float s[2] = {sum2(s1), sum2(s0)};
        join_sums<kQuads>(s, cta.scratch, flip, c.T);
        s1 = f2(-s[0] * a.inv_h), s0 = f2(-s[1] * a.inv_h);
      } else {
        float s[1] = {sum2(s1)};
        join_sums<kQuads>(s, cta.scratch, flip, c.T);
        s1 = f2(-s[0] * a.inv_h);
      }
      const F2 rr = f2(now.y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        F2 e = fma2(bh[k], s1, q[k]);
        if (LAYER) e = add2(e, s0);
        q[k] = mul2(e, rr);
      }
    }
    if (live) c.write(static_cast<A*>(a.db) + r * a.d.hidden, q);
  }
  if (a.n_sums == 0) return;
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * a.n_sums * a.d.hidden;
  const int groups = kMany ? c.n / c.T : 1;
  char* hold = cta.vec;  // the CTA's rows are done: room for its groups' sums
  if constexpr (MAP != kAny) copies_wait(0);
  auto leave = [&](int which, F2 (&v)[4]) {
    if (a.slot[which] < 0) return;
    if (groups > 1) {  // the groups' sums in order
      __syncthreads();
      for (int k = 0; k < 4; ++k) reinterpret_cast<uint64_t*>(hold)[k * c.n + c.tid] = v[k].w;
      __syncthreads();
      if (cta.group > 0) return;
      for (int g = 1; g < groups; ++g)
        for (int k = 0; k < 4; ++k) {
          F2 e;
          e.w = reinterpret_cast<uint64_t*>(hold)[k * c.n + g * c.T + c.t];
          v[k] = add2(v[k], e);
        }
    }
    c.write(mine + static_cast<int64_t>(a.slot[which]) * a.d.hidden, v);
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

// Threads of a row, and of a CTA.
inline int join_lanes(int64_t hidden) {
  if (hidden <= 64) return 8;
  if (hidden <= 128) return 16;
  return static_cast<int>((hidden + 255) / 256 * 32);
}
inline int join_threads(int64_t hidden) { return std::max(hidden <= 256 ? kJoinSmallCta : 0, join_lanes(hidden)); }

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
  l.lanes = join_lanes(a.d.hidden);
  const int T8 = join_threads(a.d.hidden) * 8;
  auto vector = [&](bool present) {
    if (!present) return -1;
    const int at = l.vec_bytes;
    l.vec_bytes += T8 * 4;
    return at;
  };
  l.w1 = vector(a.in.b != nullptr);
  l.b1 = vector(a.in.bias_post != nullptr);
  l.w2 = vector(backward ? a.d_n != nullptr : a.in.w_pre != nullptr);
  l.b2 = vector(!backward && a.in.bias_pre != nullptr);
  if (backward && l.vec_bytes == 0) l.vec_bytes = T8 * 4;  // holds the groups' sums at the end
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

template <class A, class R, bool LAYER, bool OWN, int MAP, int MAXT>
int launch_join_rows_as(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  const void* fn = backward ? reinterpret_cast<const void*>(&k_join_rows_backward<A, R, LAYER, OWN, MAP, MAXT>)
                            : reinterpret_cast<const void*>(&k_join_rows<A, R, LAYER, OWN, MAP, MAXT>);
  const int threads = join_threads(a.d.hidden), groups = threads / join_lanes(a.d.hidden);
  int fit = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, threads, 0);
  if (e != cudaSuccess) return static_cast<int>(e);
  // what the registers let run at once
  int ctas = std::max(1, std::min(fit, (backward ? kJoinThreadsBackward : kJoinThreadsForward) / threads));
  JoinLayout l = join_layout(a, static_cast<JoinMap>(MAP), backward, ctas);
  // two rows ahead before one more CTA
  while (ctas > 1 && ((MAP != kAny && l.stages < 2) || join_smem(l) > kJoinSmemMost / ctas - 1024)) {
    --ctas;
    l = join_layout(a, static_cast<JoinMap>(MAP), backward, ctas);
  }
  if ((MAP != kAny && l.stages < 1) || join_smem(l) > kJoinSmemMost) return -1;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmemMost);
  if (e != cudaSuccess) return static_cast<int>(e);
  const int64_t work = (a.d.rows + groups - 1) / groups;
  const int grid = static_cast<int>(std::min<int64_t>(work, static_cast<int64_t>(ctas) * kSMs));
  *workers = grid;
  JoinArgs copy = a;
  void* args[] = {&copy, &l};
  return static_cast<int>(cudaLaunchKernel(fn, dim3(grid), dim3(threads), args, join_smem(l), s));
}

template <class A, class R, bool LAYER, bool OWN, int MAP>
int launch_join_rows_map(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  if (a.d.hidden <= 256)
    return launch_join_rows_as<A, R, LAYER, OWN, MAP, kJoinSmallCta>(a, backward, workers, s);
  // up to 512 threads a CTA leave 128 registers a thread, 1024 leave 64
  if (join_threads(a.d.hidden) <= 512)
    return launch_join_rows_as<A, R, LAYER, OWN, MAP, 512>(a, backward, workers, s);
  return launch_join_rows_as<A, R, LAYER, OWN, MAP, 1024>(a, backward, workers, s);
}

template <class A, class R, bool LAYER, bool OWN>
int launch_join_rows_kind(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  constexpr int kWide = sizeof(A) == 2 && sizeof(R) == 2 ? kOct : kQuad;
  int e = -1;
  if (join_map<A, R>(a) != kAny) e = launch_join_rows_map<A, R, LAYER, OWN, kWide>(a, backward, workers, s);
  if (e == -1) e = launch_join_rows_map<A, R, LAYER, OWN, kAny>(a, backward, workers, s);
  return e;
}

// -1: these rows do not fit here.
template <class A, class R>
int launch_join_rows(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  if (a.d.hidden > kJoinRowMost) return -1;
  const bool own = a.d.gate_kind == ZERO_GATE_ROW || a.d.gate_kind == ZERO_GATE_FULL;
  if (a.layer)
    return own ? launch_join_rows_kind<A, R, true, true>(a, backward, workers, s)
               : launch_join_rows_kind<A, R, true, false>(a, backward, workers, s);
  return own ? launch_join_rows_kind<A, R, false, true>(a, backward, workers, s)
             : launch_join_rows_kind<A, R, false, false>(a, backward, workers, s);
}

}  // namespace zero
