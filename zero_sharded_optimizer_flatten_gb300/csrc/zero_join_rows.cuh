// The block join for rows of at most 8192 channels: a row's values stay in
// registers, 8 or 16 columns a thread, from the one read to the one write.
// Where not one row's arrays and the folded vectors fit into shared memory the
// launch is left to the element kernels of zero_join.cu: fp32 with layer norms
// on both sides and a full gate (forward above 7680 channels, backward above
// 6656), and other backward passes with seven fp32 arrays and vectors in all
// (above 7680).
//
// Row split.  Above 256 channels a CTA of whole warps takes a row at a time; a
// row's sums go through one shuffle tree a warp and one barrier.  Rows that a
// warp can hold (256 channels, 512 with 16 columns a thread) are taken by 8 to
// 32 lanes and a CTA of 128 threads has several.  Rows are handed out
// grid-stride.
//
// Column maps.  A thread's columns come in units of u neighbours, unit j of
// thread t of a row's T at column u (t + j T): u = 8 (kOct) where all rows are
// 16-bit, 16-byte accesses; u = 4 (kQuad) where a 32-bit array takes part, so
// fp32 accesses are whole 512-byte runs a warp; and for rows that start
// anywhere (odd lengths, views) u = 2 (kPair) for 16-bit rows, u = 1 (kLone)
// with 32-bit ones.
//
// Loads.  Rows are read ahead through a ring in shared memory filled by
// asynchronous copies.  kOct and kQuad: every thread copies just the columns
// that it will use, so the ring needs no barrier.  kPair and kLone: the row's
// covering 16-byte chunks are copied as they lie, with one barrier a row;
// chunks that reach outside the tensor (its first and last rows) go element
// by element.
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
constexpr int kJoinScratch = 2 * 8 * 32 * 4;  // two buffers of eight sums a warp
constexpr int kJoinSmallCta = 128;         // threads of a CTA of several rows

enum JoinMap { kOct, kQuad, kPair, kLone };

// What lies in the ring and in the vectors' part of shared memory; offsets in
// bytes, -1: absent.
struct JoinLayout {
  int32_t lanes;                    // threads of a row
  int32_t stages, stage_bytes;
  int32_t x, b, d_o, d_n, gate;     // within a stage
  int32_t w1, b1, w2, b2;           // from the vectors' start
  int32_t vec_bytes;
  // ends of the inputs: kPair and kLone read whole chunks up to there
  const char *x_end, *b_end, *do_end, *dn_end, *gate_end;
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

// A row whose covering chunks reach outside its tensor: whole chunks where
// they do not, elements of E bytes one by one where they do.
template <int E>
__device__ __noinline__ void copy_edge_row(char* row_at, const char* q, int skip, int bytes, int from, int step,
                                           const char* first, const char* end) {
#pragma unroll 1
  for (int i = from; i < skip + bytes; i += step) {
    if (q + i >= first && q + i + 16 <= end) {
      copy_async<16>(smem_of(row_at + i), q + i);
      continue;
    }
#pragma unroll 1
    for (int e = max(i, skip); e < min(i + 16, skip + bytes); e += E) {
      if constexpr (E == 4)
        *reinterpret_cast<uint32_t*>(row_at + e) = *reinterpret_cast<const uint32_t*>(q + e);
      else
        *reinterpret_cast<uint16_t*>(row_at + e) = *reinterpret_cast<const uint16_t*>(q + e);
    }
  }
}

template <class T>
__device__ __forceinline__ F2 widen2(uint32_t w) {
  float lo, hi;
  Elem<T>::unpack(w, lo, hi);
  return f2(lo, hi);
}
template <class T>
__device__ __forceinline__ uint32_t pack2(F2 v) {
  float lo, hi;
  f2_out(v, lo, hi);
  return Elem<T>::pack(lo, hi);
}

// A thread's 2 NP columns of a row; in registers they are NP pairs.
template <int MAP, int NP>
struct JoinCols {
  static constexpr bool kWide = MAP == kOct || MAP == kQuad;
  static constexpr int kUnit = MAP == kOct ? 8 : MAP == kQuad ? 4 : MAP == kPair ? 2 : 1;
  static constexpr int kUnits = 2 * NP / kUnit;
  int t, T;        // place among the row's threads
  int tid, n;      // place in the CTA: where its slots are
  int group;       // the thread's row among the CTA's
  int hidden;
  int whole;       // the thread's units that lie in the row
  bool half;       // kPair: the unit after them does with its first column
  __device__ __forceinline__ int col(int k) const { return kUnit * (t + k / kUnit * T) + k % kUnit; }
  __device__ __forceinline__ void count() {
    const int units = hidden / kUnit;
    whole = units > t ? (units - t + T - 1) / T : 0;
    half = MAP == kPair && (hidden & 1) && units >= t && (units - t) % T == 0;
  }
  __device__ __forceinline__ bool has(int k) const {
    return k / kUnit < whole || (MAP == kPair && half && k == 2 * whole);
  }
  __device__ __forceinline__ bool ragged() const { return whole < kUnits; }

  // A row's copy into its place `at` in shared memory.
  template <int TYPE>
  __device__ __forceinline__ void fetch(char* at, const void* row, const void* first, const char* end) const {
    constexpr int E = TYPE == ZERO_FP32 ? 4 : 2;
    const char* p = static_cast<const char*>(row);
    if constexpr (kWide) {
      constexpr int B = kUnit * E, W = B < 16 ? B : 16;
      const uint32_t slot = smem_of(at);
#pragma unroll
      for (int j = 0; j < kUnits; ++j)
        if (has(j * kUnit)) {
#pragma unroll
          for (int h = 0; h < B / W; ++h)
            copy_async<W>(slot + W * ((j * (B / W) + h) * n + tid), p + B * (t + j * T) + W * h);
        }
    } else {
      // chunks as they lie, the row's first byte at its own place in a chunk
      const int bytes = hidden * E, skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
      char* row_at = at + group * row_bytes(E);
      const char* q = p - skip;
      if (q >= static_cast<const char*>(first) && q + ((skip + bytes + 15) & ~15) <= end) {
        const uint32_t dst = smem_of(row_at);
        for (int i = 16 * t; i < skip + bytes; i += 16 * T) copy_async<16>(dst + i, q + i);
      } else {
        copy_edge_row<E>(row_at, q, skip, bytes, 16 * t, 16 * T, static_cast<const char*>(first), end);
      }
    }
  }
  __device__ __forceinline__ int row_bytes(int elem) const { return 2 * NP * T * elem + 16; }

  // The same row's columns, zero past its end (kWide: slots without a column
  // are cleared once).  row: where it was copied from.
  template <class E>
  __device__ __forceinline__ void read(const char* at, const void* row, F2 (&v)[NP]) const {
    constexpr int B = sizeof(E);
    if constexpr (kWide) {
      constexpr int W = kUnit * B < 16 ? 8 : 16;
#pragma unroll
      for (int j = 0; j < 2 * NP * B / W; ++j) {
        const char* p = at + W * (j * n + tid);
        if constexpr (B == 4) {
          quad32(p, v + 2 * j);
        } else if constexpr (W == 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(p);
          v[4 * j] = widen2<E>(w.x), v[4 * j + 1] = widen2<E>(w.y);
          v[4 * j + 2] = widen2<E>(w.z), v[4 * j + 3] = widen2<E>(w.w);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          v[2 * j] = widen2<E>(w.x), v[2 * j + 1] = widen2<E>(w.y);
        }
      }
    } else {
      const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
      const char* p = at + group * row_bytes(B) + skip;
      // (all the thread's columns have a place, whether the row has them or not)
      if (MAP == kPair && (skip & 3) == 0 && B == 2) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(p + 2 * col(2 * k));
          if constexpr (B == 2) v[k] = widen2<E>(has(2 * k + 1) ? w : has(2 * k) ? w & 0xffffu : 0u);
        }
      } else {
        const E* e = reinterpret_cast<const E*>(p);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float lo = Elem<E>::widen(e[col(2 * k)]), hi = Elem<E>::widen(e[col(2 * k + 1)]);
          v[k] = f2(has(2 * k) ? lo : 0.f, has(2 * k + 1) ? hi : 0.f);
        }
      }
    }
  }
  // A vector's slots: this thread's binary32 values, planes of four.
  __device__ __forceinline__ void vector_in(char* vec, const float (&f)[2 * NP]) const {
#pragma unroll
    for (int q = 0; q < NP / 2; ++q)
      *reinterpret_cast<float4*>(vec + 16 * (q * n + tid)) =
          make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  }
  __device__ __forceinline__ void vector(const char* vec, F2 (&v)[NP]) const {
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) quad32(vec + 16 * (q * n + tid), v + 2 * q);
  }
  template <class E>
  __device__ __forceinline__ void write(E* row, const F2 (&v)[NP]) const {
    if constexpr (kWide) {
      constexpr int Q = kUnit / 4;  // quads of a unit
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        if (!has(j * kUnit)) continue;
        E* p = row + col(j * kUnit);
        if constexpr (sizeof(E) == 4) {
#pragma unroll
          for (int h = 0; h < Q; ++h)
            *reinterpret_cast<ulonglong2*>(p + 4 * h) =
                make_ulonglong2(v[2 * (j * Q + h)].w, v[2 * (j * Q + h) + 1].w);
        } else if constexpr (MAP == kOct) {
          *reinterpret_cast<uint4*>(p) = make_uint4(pack2<E>(v[4 * j]), pack2<E>(v[4 * j + 1]),
                                                    pack2<E>(v[4 * j + 2]), pack2<E>(v[4 * j + 3]));
        } else {
          *reinterpret_cast<uint2*>(p) = make_uint2(pack2<E>(v[2 * j]), pack2<E>(v[2 * j + 1]));
        }
      }
    } else {
      const bool whole = MAP == kPair && sizeof(E) == 2 && (reinterpret_cast<uintptr_t>(row) & 3) == 0;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        if constexpr (MAP == kPair && sizeof(E) == 2) {
          if (whole && has(2 * k + 1)) {
            *reinterpret_cast<uint32_t*>(row + col(2 * k)) = pack2<E>(v[k]);
            continue;
          }
        }
        float lo, hi;
        f2_out(v[k], lo, hi);
        if (has(2 * k)) row[col(2 * k)] = Elem<E>::narrow(lo);
        if (has(2 * k + 1)) row[col(2 * k + 1)] = Elem<E>::narrow(hi);
      }
    }
  }
  __device__ __forceinline__ void write_any(void* row, int64_t at, int type, const F2 (&v)[NP]) const {
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

template <int NP>
__device__ __forceinline__ void clear(F2 (&v)[NP]) {
#pragma unroll
  for (int k = 0; k < NP; ++k) v[k] = f2(0.f);
}

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
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_all_sum(v[k]);
    float* part = scratch + flip * 256;
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
}

// w1, b1, w2, b2 (see above) to this thread's slots.
template <int MAP, int NP>
__device__ __forceinline__ void fold_vectors(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP, NP>& c,
                                             char* vec) {
  auto each = [&](int at, auto value) {
    if (at < 0) return;
    float f[2 * NP];
#pragma unroll
    for (int k = 0; k < 2 * NP; ++k) f[k] = c.has(k) ? value(c.col(k)) : 0.f;
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

// Where row r of an input lies.
// (Row numbers and strides fit 31 bits here, so the product is one
// instruction; their products do not.)
template <class E>
__device__ __forceinline__ const E* row_of(const void* p, int r, int64_t stride) {
  return static_cast<const E*>(p) + static_cast<int64_t>(r) * static_cast<int>(stride);
}
template <class E>
__device__ __forceinline__ E* out_row(void* p, int r, int64_t hidden) {
  return static_cast<E*>(p) + static_cast<int64_t>(r) * static_cast<int>(hidden);
}
__device__ __forceinline__ const char* gate_row_of(const JoinArgs& a, int r) {
  return static_cast<const char*>(a.in.gate) +
         static_cast<int64_t>(r) * static_cast<int>(a.d.gate_stride) * type_bytes(a.d.gate_dtype);
}

// Row r's inputs into stage `stage`.
template <class A, class R, bool OWN, int MAP, int NP>
__device__ __forceinline__ void fetch_row(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP, NP>& c,
                                          char* ring, int stage, int r) {
  if (r < static_cast<int>(a.d.rows)) {
    char* s = ring + stage * l.stage_bytes;
    c.template fetch<Elem<R>::kType>(s + l.x, row_of<R>(a.in.x, r, a.d.x_stride), a.in.x, l.x_end);
    if (l.b >= 0)
      c.template fetch<Elem<A>::kType>(s + l.b, row_of<A>(a.in.b, r, a.d.b_stride), a.in.b, l.b_end);
    if (l.d_o >= 0)
      c.template fetch<Elem<R>::kType>(s + l.d_o, row_of<R>(a.d_o, r, a.d.do_stride), a.d_o, l.do_end);
    if (l.d_n >= 0)
      c.template fetch<Elem<A>::kType>(s + l.d_n, row_of<A>(a.d_n, r, a.d.dn_stride), a.d_n, l.dn_end);
    if (OWN && l.gate >= 0) {
      if (a.d.gate_dtype == ZERO_FP32)
        c.template fetch<ZERO_FP32>(s + l.gate, gate_row_of(a, r), a.in.gate, l.gate_end);
      else
        c.template fetch<ZERO_BF16>(s + l.gate, gate_row_of(a, r), a.in.gate, l.gate_end);  // or fp16
    }
  }
  copies_commit();
}

// A row's own gate (1 without one), loaded a row ahead.
template <bool OWN>
__device__ __forceinline__ float own_gate(const JoinArgs& a, int r) {
  if (!OWN || a.d.gate_kind != ZERO_GATE_ROW || r >= static_cast<int>(a.d.rows)) return 1.f;
  return load_any(a.in.gate, static_cast<int64_t>(r) * static_cast<int>(a.d.gate_stride), a.d.gate_dtype);
}

// y w1: what multiplies the normalised block output, and y itself where rows
// (`own`) or elements have their own gates (OWN).
template <class A, bool OWN, int MAP, int NP>
__device__ __forceinline__ void row_gate(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP, NP>& c,
                                         const char* stage, const char* vec, int r, float own, F2 (&y)[NP],
                                         F2 (&w)[NP]) {
  c.vector(vec + l.w1, w);
  if constexpr (OWN) {
    if (a.d.gate_kind == ZERO_GATE_FULL) {
      if (a.d.gate_dtype == ZERO_FP32)
        c.template read<float>(stage + l.gate, gate_row_of(a, r), y);
      else
        c.template read<A>(stage + l.gate, gate_row_of(a, r), y);
    } else {
      const F2 one = f2(own);
#pragma unroll
      for (int k = 0; k < NP; ++k) y[k] = one;
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) w[k] = mul2(w[k], y[k]);
  }
}

// The ring's step at the start of row i: its copies have arrived, and the
// slots of the row before it are free for the row `stages` behind that one.
// kWide refills its own slots later, when it has read them.
template <class A, class R, bool OWN, bool MANY, int MAP, int NP>
__device__ __forceinline__ void ring_step(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP, NP>& c,
                                          char* ring, int stage, int r, int step) {
  auto meet = [] {  // the threads of a row
    if constexpr (MANY)
      __syncwarp();
    else
      __syncthreads();
  };
  if constexpr (JoinCols<MAP, NP>::kWide) {
    copies_wait(l.stages - 1);
  } else if (l.stages == 1) {
    meet();
    fetch_row<A, R, OWN>(a, l, c, ring, 0, r);
    copies_wait(0);
    meet();
  } else {
    copies_wait(l.stages - 2);
    meet();
    const int free = stage == 0 ? l.stages - 1 : stage - 1;
    fetch_row<A, R, OWN>(a, l, c, ring, free, r + (l.stages - 1) * step);
  }
}
template <class A, class R, bool OWN, int MAP, int NP>
__device__ __forceinline__ void ring_start(const JoinArgs& a, const JoinLayout& l, const JoinCols<MAP, NP>& c,
                                           char* ring, int r, int step) {
  const int ahead = JoinCols<MAP, NP>::kWide ? l.stages : l.stages - 1;
  for (int s = 0; s < ahead; ++s) fetch_row<A, R, OWN>(a, l, c, ring, s, r + s * step);
}

// Mean (layer only) and 1/deviation of a row; v becomes the normalised row.
template <bool LAYER, int QUADS, int MAP, int NP>
__device__ __forceinline__ void normalise(const JoinArgs& a, const JoinCols<MAP, NP>& c, float* scratch,
                                          int& flip, F2 (&v)[NP], float& mean, float& r) {
  mean = 0.f;
  if constexpr (LAYER) {
    F2 q = v[0];
#pragma unroll
    for (int k = 1; k < NP; ++k) q = add2(q, v[k]);
    float s[1] = {sum2(q)};
    join_sums<QUADS>(s, scratch, flip, c.T);
    mean = s[0] * a.inv_h;
    const F2 m = f2(-mean);
#pragma unroll
    for (int k = 0; k < NP; ++k) v[k] = add2(v[k], m);
    if (c.ragged()) {
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        float lo, hi;
        f2_out(v[k], lo, hi);
        v[k] = f2(c.has(2 * k) ? lo : 0.f, c.has(2 * k + 1) ? hi : 0.f);
      }
    }
  }
  F2 q = mul2(v[0], v[0]), p = mul2(v[1], v[1]);
#pragma unroll
  for (int k = 2; k < NP; k += 2) q = fma2(v[k], v[k], q), p = fma2(v[k + 1], v[k + 1], p);
  float s[1] = {sum2(add2(q, p))};
  join_sums<QUADS>(s, scratch, flip, c.T);
  r = rsqrtf(fmaf(s[0], a.inv_h, a.eps));
  const F2 rr = f2(r);
#pragma unroll
  for (int k = 0; k < NP; ++k) v[k] = mul2(v[k], rr);
}

// What both kernels set up.
template <int MAP, int NP, bool MANY>
struct JoinCta {
  float* scratch;
  char *vec, *ring;
  JoinCols<MAP, NP> c;
  int first, step, rows;  // the CTA's rows: first + group + i * step, while first + i * step is one
  __device__ __forceinline__ JoinCta(const JoinArgs& a, const JoinLayout& l, char* smem) {
    scratch = reinterpret_cast<float*>(smem);
    vec = smem + kJoinScratch;
    ring = vec + l.vec_bytes;
    const int tid = static_cast<int>(threadIdx.x), n = static_cast<int>(blockDim.x);
    const int groups = MANY ? n / l.lanes : 1;
    c.group = MANY ? tid / l.lanes : 0;
    c.t = MANY ? tid % l.lanes : tid, c.T = MANY ? l.lanes : n, c.tid = tid, c.n = n;
    c.hidden = static_cast<int>(a.d.hidden);
    c.count();
    first = static_cast<int>(blockIdx.x) * groups;
    step = static_cast<int>(gridDim.x) * groups;
    rows = static_cast<int>(a.d.rows);
    // sums of warps the CTA lacks, and slots of columns a row lacks
    for (int i = tid; i < kJoinScratch / 4; i += n) scratch[i] = 0.f;
    if constexpr (JoinCols<MAP, NP>::kWide)
      for (int i = tid; i < l.stages * l.stage_bytes / 16; i += n)
        reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
};

// Measured, us and share of a plain copy's bandwidth: 16384 x 4096 bf16, norms
// on both sides, channel gate, 94 (0.84); the same with layer norms 118 (0.67),
// four dependent sums a row; 8191 x 5120, pre norm alone on an fp32 stream, 89
// (0.83).  Bound by HBM but for layer norms and short rows.
template <class A, class R, bool LAYER, bool OWN, int MAP, int MAXT, int NP>
__global__ void __launch_bounds__(MAXT, NP == 4 ? kJoinThreadsForward / MAXT : 512 / MAXT) k_join_rows(
    const __grid_constant__ JoinArgs a, const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  constexpr bool kMany = MAXT == kJoinSmallCta;  // several rows a CTA
  constexpr int kQuads = MAXT / 128;              // a row's warps in fours
  constexpr bool kWide = JoinCols<MAP, NP>::kWide;
  JoinCta<MAP, NP, kMany> cta(a, l, smem);
  const JoinCols<MAP, NP>& c = cta.c;
  int flip = 0, stage = 0;
  ring_start<A, R, OWN>(a, l, c, cta.ring, cta.first + c.group, cta.step);
  fold_vectors(a, l, c, cta.vec);
  float next_own = own_gate<OWN>(a, cta.first + c.group);
  for (int base = cta.first; base < cta.rows; base += cta.step) {
    const float own = next_own;
    next_own = own_gate<OWN>(a, base + c.group + cta.step);
    // a group past the last row works on it once more and writes nothing
    const int r = kMany ? min(base + c.group, cta.rows - 1) : base;
    const bool live = !kMany || base + c.group < cta.rows;
    ring_step<A, R, OWN, kMany>(a, l, c, cta.ring, stage, base + c.group, cta.step);
    const char* in = cta.ring + stage * l.stage_bytes;
    F2 o[NP];
    float mb = 0.f, rb = 1.f, mo = 0.f, ro = 1.f;
    c.template read<R>(in + l.x, row_of<R>(a.in.x, r, a.d.x_stride), o);
    if (a.in.b) {
      F2 v[NP], y[NP], w[NP];
      c.template read<A>(in + l.b, row_of<A>(a.in.b, r, a.d.b_stride), v);
      if (a.in.w_post) normalise<LAYER, kQuads>(a, c, cta.scratch, flip, v, mb, rb);
      row_gate<A, OWN>(a, l, c, in, cta.vec, r, own, y, w);
#pragma unroll
      for (int k = 0; k < NP; ++k) o[k] = fma2(w[k], v[k], o[k]);
      if (LAYER && l.b1 >= 0) {
        c.vector(cta.vec + l.b1, w);
#pragma unroll
        for (int k = 0; k < NP; ++k) o[k] = OWN ? fma2(w[k], y[k], o[k]) : add2(w[k], o[k]);
      }
    }
    // this thread has read its slots of the stage: the row `stages` ahead
    if constexpr (kWide) fetch_row<A, R, OWN>(a, l, c, cta.ring, stage, base + c.group + l.stages * cta.step);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
    if (a.o && live) c.write(out_row<R>(a.o, r, a.d.hidden), o);
    if (a.in.w_pre) {
      normalise<LAYER, kQuads>(a, c, cta.scratch, flip, o, mo, ro);
      if (a.n && live) {
        F2 w[NP];
        c.vector(cta.vec + l.w2, w);
        if (LAYER && l.b2 >= 0) {
          F2 d[NP];
          c.vector(cta.vec + l.b2, d);
#pragma unroll
          for (int k = 0; k < NP; ++k) o[k] = fma2(o[k], w[k], d[k]);
        } else {
#pragma unroll
          for (int k = 0; k < NP; ++k) o[k] = mul2(o[k], w[k]);
        }
        c.write(out_row<A>(a.n, r, a.d.hidden), o);
      }
    }
    if (a.stats && live && c.t == 0) a.stats[r] = make_float4(mb, rb, mo, ro);
  }
}

// Totals over a row's lanes (of a warp) of N values, N a power of two and at
// most the lanes: lane (lanes / N) k of the row holds value k's.  Halves are
// exchanged while a lane has several values, so eight values take 9 shuffles
// over 32 lanes and not 40.
template <int N>
__device__ __forceinline__ float scatter_sums(float (&v)[N], int lanes) {
  const int lane = threadIdx.x & 31;
  int o = lanes >> 1;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[i + n] : v[i], send = upper ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
  }
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(kFull, v[0], o);
  return v[0];
}

// join_sums for 4 or 8 values.
template <int QUADS, int N>
__device__ __forceinline__ void join_many_sums(float (&v)[N], float* scratch, int& flip, int lanes) {
  const int lane = threadIdx.x & 31;
  if constexpr (QUADS == 1) {
    const float total = scatter_sums(v, lanes);
    const int first = lane & ~(lanes - 1), apart = lanes / N;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(kFull, total, first + k * apart);
  } else {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float* part = scratch + flip * 256;
    flip ^= 1;
    const float mine = scatter_sums(v, 32);
    if (lane % (32 / N) == 0) part[warp * N + lane / (32 / N)] = mine;
    __syncthreads();
    const float4* p = reinterpret_cast<const float4*>(part + lane * N);
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const float4 q = lane < warps ? p[k / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
      v[k] = q.x, v[k + 1] = q.y, v[k + 2] = q.z, v[k + 3] = q.w;
    }
    const float total = scatter_sums(v, 32);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(kFull, total, k * (32 / N));
  }
}

// The backward pass of a row in one round of sums.  With e = w1 bh (the
// block's part of o without its own gate), h = oh and g' = do + R_o t, the
// gradient of o is go = g' - R_o (mean(t) + h mean(t h)), so the sums over go
// that the post norm needs follow from sums over g':
//   sum e go = sum e g' - R_o mean(t) sum e - R_o mean(t h) sum e h,
// and the same with w1 in place of e (layer only, as mean(t) is).  One barrier
// a row in place of two, and less to hold across it: 8192 x 8192 bf16 200 ->
// 145 us, where the registers counted; 16384 x 4096 stayed at 155.
//
// Measured, us and share of a plain copy's bandwidth: 16384 x 4096 bf16, norms
// on both sides, channel gate, 154 (0.77); 8192 x 8192 144 (0.83); 8192 x 4096
// fp32 with a full gate 194 (0.82).  Long rows are bound by HBM, short ones and
// layer norms (eight sums a row, 16384 x 4096 194) by instructions.
template <class A, class R, bool LAYER, bool OWN, int MAP, int MAXT, int NP>
__global__ void __launch_bounds__(MAXT, MAXT == kJoinSmallCta ? 4 : 1) k_join_rows_backward(
    const __grid_constant__ JoinArgs a, const __grid_constant__ JoinLayout l) {
  extern __shared__ __align__(16) char smem[];
  constexpr bool kMany = MAXT == kJoinSmallCta;  // several rows a CTA
  constexpr int kQuads = MAXT / 128;              // a row's warps in fours
  constexpr bool kWide = JoinCols<MAP, NP>::kWide;
  let_next_start();  // the column sums' launch
  JoinCta<MAP, NP, kMany> cta(a, l, smem);
  const JoinCols<MAP, NP>& c = cta.c;
  int flip = 0, stage = 0;
  ring_start<A, R, OWN>(a, l, c, cta.ring, cta.first + c.group, cta.step);
  fold_vectors(a, l, c, cta.vec);
  const bool full = OWN && a.d.gate_kind == ZERO_GATE_FULL, post = a.in.w_post != nullptr;
  F2 P[NP], Q[NP], S[NP], B[NP];
  clear(P), clear(Q), clear(S), clear(B);
  float4 st = make_float4(0.f, 1.f, 0.f, 1.f);
  if (a.stats && cta.first < cta.rows) st = __ldg(a.stats + min(cta.first + c.group, cta.rows - 1));
  float next_own = own_gate<OWN>(a, cta.first + c.group);
  for (int base = cta.first; base < cta.rows; base += cta.step) {
    const float own = next_own;
    next_own = own_gate<OWN>(a, base + c.group + cta.step);
    const int r = kMany ? min(base + c.group, cta.rows - 1) : base;
    const bool live = !kMany || base + c.group < cta.rows;
    const float4 now = st;
    if (a.stats) st = __ldg(a.stats + min(r + cta.step, cta.rows - 1));  // the next row's
    ring_step<A, R, OWN, kMany>(a, l, c, cta.ring, stage, base + c.group, cta.step);
    const char* in = cta.ring + stage * l.stage_bytes;
    F2 go[NP], bh[NP], y[NP], oh[NP];
    // sums: t oh, e g', e oh; t, w1 g', w1 oh, e, w1 (layer)
    constexpr int N = LAYER ? 8 : 4;
    float s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = 0.f;
    clear(oh);
    if (a.d_o)
      c.template read<R>(in + l.d_o, row_of<R>(a.d_o, r, a.d.do_stride), go);
    else
      clear(go);
    if (a.in.b) {
      c.template read<A>(in + l.b, row_of<A>(a.in.b, r, a.d.b_stride), bh);
      if (post) {
        const F2 rr = f2(now.y), m = f2(-now.x);
#pragma unroll
        for (int k = 0; k < NP; ++k) bh[k] = mul2(LAYER ? add2(bh[k], m) : bh[k], rr);
      }
      if (OWN) {
        if (!full) {
          const F2 one = f2(own);
#pragma unroll
          for (int k = 0; k < NP; ++k) y[k] = one;
        } else if (a.d.gate_dtype == ZERO_FP32) {
          c.template read<float>(in + l.gate, gate_row_of(a, r), y);
        } else {
          c.template read<A>(in + l.gate, gate_row_of(a, r), y);
        }
      }
    }
    if (a.d_n) {
      F2 t[NP], w[NP];
      c.template read<R>(in + l.x, row_of<R>(a.in.x, r, a.d.x_stride), oh);
      c.template read<A>(in + l.d_n, row_of<A>(a.d_n, r, a.d.dn_stride), t);
      if (a.in.b) {
        c.vector(cta.vec + l.w1, w);
#pragma unroll
        for (int k = 0; k < NP; ++k) oh[k] = fma2(OWN ? mul2(w[k], y[k]) : w[k], bh[k], oh[k]);
        if (LAYER && l.b1 >= 0) {
          c.vector(cta.vec + l.b1, w);
#pragma unroll
          for (int k = 0; k < NP; ++k) oh[k] = OWN ? fma2(w[k], y[k], oh[k]) : add2(w[k], oh[k]);
        }
      }
      c.vector(cta.vec + l.w2, w);
      const F2 rr = f2(now.w), m = f2(-now.z);
      F2 s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        oh[k] = mul2(LAYER ? add2(oh[k], m) : oh[k], rr);
        if (live) {
          P[k] = fma2(t[k], oh[k], P[k]);
          if (LAYER) Q[k] = add2(Q[k], t[k]);
        }
        t[k] = mul2(t[k], w[k]);  // zero past the row's end, as dn and w2 are
        s1 = fma2(t[k], oh[k], s1);
        if (LAYER) s0 = add2(s0, t[k]);
        go[k] = fma2(t[k], rr, go[k]);
      }
      s[0] = sum2(s1);
      if constexpr (LAYER) s[3] = sum2(s0);
    }
    // every input has been read: the row `stages` ahead
    if constexpr (kWide) fetch_row<A, R, OWN>(a, l, c, cta.ring, stage, base + c.group + l.stages * cta.step);
    stage = stage + 1 == l.stages ? 0 : stage + 1;
    if (a.in.b && (post || OWN)) {
      F2 w[NP], t1 = f2(0.f), t2 = f2(0.f), t4 = f2(0.f), t5 = f2(0.f), t6 = f2(0.f), t7 = f2(0.f);
      c.vector(cta.vec + l.w1, w);  // zero past the row's end
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        if (full) w[k] = mul2(w[k], y[k]);
        const F2 e = mul2(w[k], bh[k]);
        t1 = fma2(e, go[k], t1);
        t2 = fma2(e, oh[k], t2);
        if constexpr (LAYER) {
          t4 = fma2(w[k], go[k], t4);
          t5 = fma2(w[k], oh[k], t5);
          t6 = add2(t6, e);
          t7 = add2(t7, w[k]);
        }
      }
      s[1] = sum2(t1), s[2] = sum2(t2);
      if constexpr (LAYER) s[4] = sum2(t4), s[5] = sum2(t5), s[6] = sum2(t6), s[7] = sum2(t7);
    }
    if (post || OWN) {
      join_many_sums<kQuads>(s, cta.scratch, flip, c.T);
    } else if (a.d_n) {  // only the sums over t
      float t[LAYER ? 2 : 1];
      t[0] = s[0];
      if constexpr (LAYER) t[1] = s[3];
      join_sums<kQuads>(t, cta.scratch, flip, c.T);
      s[0] = t[0];
      if constexpr (LAYER) s[3] = t[1];
    }
    // -R_o mean(t h) and -R_o mean(t)
    const float q1 = -now.w * (s[0] * a.inv_h), q0 = LAYER ? -now.w * (s[3 % N] * a.inv_h) : 0.f;
    if (a.d_n) {
      const F2 m1 = f2(q1), m0 = f2(q0);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        go[k] = fma2(oh[k], m1, go[k]);
        if (LAYER) go[k] = add2(go[k], m0);
      }
    }
    if (a.dx && live) c.write(out_row<R>(a.dx, r, a.d.hidden), go);
    if (!a.in.b) continue;
    if (live) {
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const F2 yg = OWN ? mul2(y[k], go[k]) : go[k];
        S[k] = fma2(yg, bh[k], S[k]);
        if (LAYER) B[k] = add2(B[k], yg);
      }
    }
    // sums over the gradient of o: e go, and w1 go
    float e_go = fmaf(q1, s[2], s[1]), w_go = 0.f;
    if constexpr (LAYER) {
      e_go = fmaf(q0, s[6], e_go);
      w_go = fmaf(q0, s[7], fmaf(q1, s[5], s[4]));
    }
    if constexpr (OWN) {
      if (a.dgate) {
        F2 u[NP], w[NP];
        if (full) {
          c.vector(cta.vec + l.w1, w);
#pragma unroll
          for (int k = 0; k < NP; ++k) u[k] = mul2(w[k], bh[k]);
          if (LAYER && l.b1 >= 0) {
            c.vector(cta.vec + l.b1, w);
#pragma unroll
            for (int k = 0; k < NP; ++k) u[k] = add2(u[k], w[k]);
          }
#pragma unroll
          for (int k = 0; k < NP; ++k) u[k] = mul2(u[k], go[k]);
          if (live) c.write_any(a.dgate, static_cast<int64_t>(r) * static_cast<int>(a.d.hidden), a.d.gate_dtype, u);
        } else {
          float d[1] = {0.f};
          if (LAYER && l.b1 >= 0) {  // b1 go over the row
            F2 t = f2(0.f);
            c.vector(cta.vec + l.b1, w);
#pragma unroll
            for (int k = 0; k < NP; ++k) t = fma2(w[k], go[k], t);
            d[0] = sum2(t);
            join_sums<kQuads>(d, cta.scratch, flip, c.T);
          }
          if (live && c.t == 0) store_any(a.dgate, r, a.d.gate_dtype, e_go + d[0]);
        }
      }
    }
    if (!a.db) continue;
    F2 w[NP];
    c.vector(cta.vec + l.w1, w);
#pragma unroll
    for (int k = 0; k < NP; ++k) go[k] = mul2(OWN ? mul2(w[k], y[k]) : w[k], go[k]);  // the gradient of N(b)
    if (post) {
      const float by = OWN && !full ? own : 1.f;  // an element's gate is in the sums
      const F2 rr = f2(now.y), m1 = f2(-by * e_go * a.inv_h), m0 = f2(-by * w_go * a.inv_h);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        F2 e = fma2(bh[k], m1, go[k]);
        if (LAYER) e = add2(e, m0);
        go[k] = mul2(e, rr);
      }
    }
    if (live) c.write(out_row<A>(a.db, r, a.d.hidden), go);
  }
  copies_wait(0);
  if (a.n_sums == 0) return;
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * a.n_sums * a.d.hidden;
  const int groups = kMany ? c.n / c.T : 1;
  char* hold = cta.vec;  // the CTA's rows are done: room for its groups' sums
  auto leave = [&](int which, F2 (&v)[NP]) {
    if (a.slot[which] < 0) return;
    if constexpr (kMany) {  // the groups' sums in order
      __syncthreads();
      for (int k = 0; k < NP; ++k) reinterpret_cast<uint64_t*>(hold)[k * c.n + c.tid] = v[k].w;
      __syncthreads();
      if (c.group > 0) return;
      for (int g = 1; g < groups; ++g)
        for (int k = 0; k < NP; ++k) {
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

// Columns of a thread, 8 or 16.  16 halve what a row costs beside its columns
// and take twice the registers.  Measured, bf16, us with 8 and with 16:
//                              forward           backward
//   65536 x 256, rms           31.8 -> 28.1      49.0 -> 49.9
//   65536 x 256, layer norms   40.4 -> 33.9      62 -> 105
//   65536 x 512, layer norms   69 -> 57          102 -> 183
//   16384 x 4096, rms          94 -> 102         156 -> 153
//   16384 x 4096, layer norms  135 -> 118        195 -> 309
//   8192 x 8192, rms           107 -> 93         267 -> 145
//   8192 x 8192, layer norms                     277 -> 240
//   8001 x 4097, rms           141 -> 102        206 -> 211
// (up to 512 channels 16 columns let a warp hold a row, without a barrier; up
// to 8192, 16 keep a CTA within 512 threads and its registers).  Shorter rows
// that start anywhere keep 8: their element accesses need the threads.
inline int join_columns(const zero_join_desc& d, bool wide, bool backward) {
  if (d.hidden > kJoinNarrow) return wide || !backward ? 16 : 8;
  if (!wide || backward) return 8;
  return d.hidden <= 512 || (d.kind == ZERO_JOIN_LAYER && d.hidden > kJoinNarrowLayer) ? 16 : 8;
}

// Threads of a row, and of a CTA.
inline int join_lanes(const zero_join_desc& d, bool wide, bool backward) {
  const int64_t hidden = d.hidden, warp = 32 * join_columns(d, wide, backward);
  if (hidden * 4 <= warp) return 8;
  if (hidden * 2 <= warp) return 16;
  return static_cast<int>((hidden + warp - 1) / warp * 32);
}
inline int join_threads(const zero_join_desc& d, bool wide, bool backward) {
  const int lanes = join_lanes(d, wide, backward);
  return lanes <= 32 ? kJoinSmallCta : lanes;
}

inline bool join_row_fits(const void* p, int64_t stride, int type, bool oct) {
  if (!p) return true;
  const int bytes = type_bytes(type);
  const int unit = oct || bytes == 4 ? 16 : 8;
  return aligned_to(p, unit) && stride * bytes % unit == 0;
}

// Whether pointers and strides allow whole 16-byte (kQuad: 8-byte) accesses.
template <class A, class R>
bool join_wide(const JoinArgs& a) {
  const zero_join_desc& d = a.d;
  const bool oct = sizeof(A) == 2 && sizeof(R) == 2;
  const int64_t H = d.hidden;
  if (H % (oct ? 8 : 4)) return false;
  auto ok = [&](const void* p, int64_t stride, int type) { return join_row_fits(p, stride, type, oct); };
  const bool full = d.gate_kind == ZERO_GATE_FULL;
  return ok(a.in.x, d.x_stride, d.res_dtype) && ok(a.in.b, d.b_stride, d.act_dtype) &&
         ok(a.d_o, d.do_stride, d.res_dtype) && ok(a.d_n, d.dn_stride, d.act_dtype) &&
         ok(a.o, H, d.res_dtype) && ok(a.n, H, d.act_dtype) && ok(a.dx, H, d.res_dtype) &&
         ok(a.db, H, d.act_dtype) &&
         (!full || (ok(a.in.gate, d.gate_stride, d.gate_dtype) && ok(a.dgate, H, d.gate_dtype)));
}

inline JoinLayout join_layout(const JoinArgs& a, bool wide, bool backward, int ctas) {
  JoinLayout l = {};
  const zero_join_desc& d = a.d;
  l.lanes = join_lanes(d, wide, backward);
  const int threads = join_threads(d, wide, backward), slots = threads * join_columns(d, wide, backward);
  auto vector = [&](bool present) {
    if (!present) return -1;
    const int at = l.vec_bytes;
    l.vec_bytes += slots * 4;
    return at;
  };
  l.w1 = vector(a.in.b != nullptr);
  l.b1 = vector(a.in.bias_post != nullptr);
  l.w2 = vector(backward ? a.d_n != nullptr : a.in.w_pre != nullptr);
  l.b2 = vector(!backward && a.in.bias_pre != nullptr);
  if (backward && l.vec_bytes == 0) l.vec_bytes = slots * 4;  // holds the groups' sums at the end
  auto row = [&](const void* p, int type, int64_t stride, const char** end) {
    if (!p) return -1;
    const int at = l.stage_bytes, bytes = type_bytes(type);
    l.stage_bytes += slots * bytes + (wide ? 0 : 16 * (threads / l.lanes));  // room for a row's offset
    *end = static_cast<const char*>(p) + ((d.rows - 1) * stride + d.hidden) * bytes;
    return at;
  };
  l.x = row(a.in.x, d.res_dtype, d.x_stride, &l.x_end);
  l.b = row(a.in.b, d.act_dtype, d.b_stride, &l.b_end);
  l.d_o = row(a.d_o, d.res_dtype, d.do_stride, &l.do_end);
  l.d_n = row(a.d_n, d.act_dtype, d.dn_stride, &l.dn_end);
  l.gate = row(d.gate_kind == ZERO_GATE_FULL ? a.in.gate : nullptr, d.gate_dtype, d.gate_stride, &l.gate_end);
  const int room = kJoinSmemMost / ctas - 1024 - kJoinScratch - l.vec_bytes;
  l.stages = std::max(0, std::min(kJoinStagesMost, room / l.stage_bytes));
  return l;
}

inline int join_smem(const JoinLayout& l) { return kJoinScratch + l.vec_bytes + l.stages * l.stage_bytes; }

inline int launch_join_rows_fn(const void* fn, KernelFacts& facts, const JoinArgs& a, bool wide, bool backward,
                               int* workers, cudaStream_t s) {
  const int threads = join_threads(a.d, wide, backward);
  const int groups = threads / join_lanes(a.d, wide, backward);
  int fit = 0;
  cudaError_t e = facts.ctas_of(fn, threads, &fit);
  if (e != cudaSuccess) return static_cast<int>(e);
  int ctas = std::max(1, std::min(fit, (backward ? kJoinThreadsBackward : kJoinThreadsForward) / threads));
  JoinLayout l = join_layout(a, wide, backward, ctas);
  while (ctas > 1 && l.stages < 2) l = join_layout(a, wide, backward, --ctas);  // a row ahead before one more CTA
  if (l.stages < 1) return -1;
  e = facts.allow(fn, join_smem(l), kJoinSmemMost);
  if (e != cudaSuccess) return static_cast<int>(e);
  const int64_t work = (a.d.rows + groups - 1) / groups;
  const int grid = static_cast<int>(std::min<int64_t>(work, static_cast<int64_t>(ctas) * kSMs));
  *workers = grid;
  JoinArgs copy = a;
  void* args[] = {&copy, &l};
  return static_cast<int>(cudaLaunchKernel(fn, dim3(grid), dim3(threads), args, join_smem(l), s));
}

template <class A, class R, bool LAYER, bool OWN, bool BACKWARD, int MAP, int MAXT, int NP>
int launch_join_rows_as(const JoinArgs& a, int* workers, cudaStream_t s) {
  static KernelFacts facts;
  const void* fn;
  if constexpr (BACKWARD)
    fn = reinterpret_cast<const void*>(&k_join_rows_backward<A, R, LAYER, OWN, MAP, MAXT, NP>);
  else
    fn = reinterpret_cast<const void*>(&k_join_rows<A, R, LAYER, OWN, MAP, MAXT, NP>);
  return launch_join_rows_fn(fn, facts, a, JoinCols<MAP, NP>::kWide, BACKWARD, workers, s);
}

template <class A, class R, bool LAYER, bool OWN, bool BACKWARD, int MAP>
int launch_join_rows_map(const JoinArgs& a, int* workers, cudaStream_t s) {
  constexpr bool wide = JoinCols<MAP, 4>::kWide;
  if (join_lanes(a.d, wide, BACKWARD) <= 32)  // short rows, as join_columns has them
    return launch_join_rows_as<A, R, LAYER, OWN, BACKWARD, MAP, kJoinSmallCta, wide && !BACKWARD ? 8 : 4>(a, workers,
                                                                                                          s);
  if constexpr (wide || !BACKWARD) {
    if (join_columns(a.d, wide, BACKWARD) == 16)
      return launch_join_rows_as<A, R, LAYER, OWN, BACKWARD, MAP, 512, 8>(a, workers, s);
  } else if (join_threads(a.d, wide, BACKWARD) > 512) {
    return launch_join_rows_as<A, R, LAYER, OWN, BACKWARD, MAP, 1024, 4>(a, workers, s);
  }
  return launch_join_rows_as<A, R, LAYER, OWN, BACKWARD, MAP, 512, 4>(a, workers, s);
}

template <class A, class R, bool LAYER, bool OWN>
int launch_join_rows_kind(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  constexpr bool k16 = sizeof(A) == 2 && sizeof(R) == 2;
  constexpr int kWide = k16 ? kOct : kQuad, kAny = k16 ? kPair : kLone;
  if (join_wide<A, R>(a))
    return backward ? launch_join_rows_map<A, R, LAYER, OWN, true, kWide>(a, workers, s)
                    : launch_join_rows_map<A, R, LAYER, OWN, false, kWide>(a, workers, s);
  return backward ? launch_join_rows_map<A, R, LAYER, OWN, true, kAny>(a, workers, s)
                  : launch_join_rows_map<A, R, LAYER, OWN, false, kAny>(a, workers, s);
}

// -1: these rows do not fit here.
template <class A, class R>
int launch_join_rows(const JoinArgs& a, bool backward, int* workers, cudaStream_t s) {
  const zero_join_desc& d = a.d;
  constexpr int64_t kMost = INT64_C(1) << 30;
  if (d.hidden > kJoinRowMost || d.rows > kMost || d.x_stride > kMost || d.b_stride > kMost ||
      d.gate_stride > kMost || d.do_stride > kMost || d.dn_stride > kMost)
    return -1;
  const bool own = a.d.gate_kind == ZERO_GATE_ROW || a.d.gate_kind == ZERO_GATE_FULL;
  if (a.layer)
    return own ? launch_join_rows_kind<A, R, true, true>(a, backward, workers, s)
               : launch_join_rows_kind<A, R, true, false>(a, backward, workers, s);
  return own ? launch_join_rows_kind<A, R, false, true>(a, backward, workers, s)
             : launch_join_rows_kind<A, R, false, false>(a, backward, workers, s);
}

}  // namespace zero
