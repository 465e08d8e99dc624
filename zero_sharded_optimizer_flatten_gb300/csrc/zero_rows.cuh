// Element access and small reductions shared by the kernels that work on
// rows of activations and on lists of gradient tensors.  Values are widened
// to binary32 on load and rounded once, to nearest even, on store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "zero.h"

namespace zero {

constexpr int kSMs = 152;  // SMs of a GB300: persistent grids are multiples of it
constexpr unsigned kFull = 0xffffffffu;

// One element and eight consecutive elements ("an octet"; 16 bytes of 16-bit
// data, 32 bytes of fp32 data, the address 16-byte aligned).
template <class T>
struct Elem;

template <>
struct Elem<float> {
  static constexpr zero_dtype kType = ZERO_FP32;
  static __device__ __forceinline__ float widen(float x) { return x; }
  static __device__ __forceinline__ float narrow(float x) { return x; }
  static __device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

template <>
struct Elem<__half> {
  static constexpr zero_dtype kType = ZERO_FP16;
  static __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x, hi = f.y;
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
  }
};

template <>
struct Elem<__nv_bfloat16> {
  static constexpr zero_dtype kType = ZERO_BF16;
  static __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
  }
};

// An octet as it was loaded: whole 16-byte chunks, widened when it is used,
// so that the loads of a thread's octets go out together.
template <class T>
struct Octet {
  static constexpr int kChunks = sizeof(T) == 4 ? 2 : 1;
  uint4 w[kChunks];
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w[0].x), v[1] = __uint_as_float(w[0].y);
      v[2] = __uint_as_float(w[0].z), v[3] = __uint_as_float(w[0].w);
      v[4] = __uint_as_float(w[1].x), v[5] = __uint_as_float(w[1].y);
      v[6] = __uint_as_float(w[1].z), v[7] = __uint_as_float(w[1].w);
    } else {
      Elem<T>::unpack(w[0].x, v[0], v[1]), Elem<T>::unpack(w[0].y, v[2], v[3]);
      Elem<T>::unpack(w[0].z, v[4], v[5]), Elem<T>::unpack(w[0].w, v[6], v[7]);
    }
  }
  __device__ __forceinline__ void load(const T* p) {  // 16-byte aligned
#pragma unroll
    for (int k = 0; k < kChunks; ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) reinterpret_cast<uint4*>(p)[k] = w[k];
  }
};

// Element i of an array whose type is known only at run time (parameters,
// gates, weights: read rarely, the branch is uniform).
__device__ __forceinline__ float load_any(const void* p, int64_t i, int type) {
  if (type == ZERO_FP32) return static_cast<const float*>(p)[i];
  if (type == ZERO_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_any(void* p, int64_t i, int type, float v) {
  if (type == ZERO_FP32)
    static_cast<float*>(p)[i] = v;
  else if (type == ZERO_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__host__ __device__ __forceinline__ int type_bytes(int type) { return type == ZERO_FP32 ? 4 : 2; }

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

// Sum over the warp, the same value in every lane (a fixed butterfly).
template <class V>
__device__ __forceinline__ V warp_all_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The launch that follows may start its CTAs; they wait for this grid's end.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Host: launch fn; early: its CTAs may start before the launch ahead of it has
// ended (they call wait_for_previous before they read what it wrote).
inline cudaError_t launch_maybe_early(const void* fn, dim3 grid, dim3 block, void** args, bool early,
                                      cudaStream_t s) {
  if (!early) return cudaLaunchKernel(fn, grid, block, args, 0, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// What a kernel was told or asked once: for each CTA size the CTAs of an SM
// that its registers allow, and whether it may use `most` bytes of shared
// memory (a driver call each, 1 us beside a launch of 4).  Devices have one
// set each, up to kDevices; beyond, every call asks.
struct KernelFacts {
  static constexpr int kDevices = 8, kSizes = 33;  // CTA sizes in warps
  std::atomic<int> fit[kDevices][kSizes];
  std::atomic<bool> large[kDevices];

  cudaError_t ctas_of(const void* fn, int threads, int* ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>* slot = dev < kDevices ? &fit[dev][threads / 32] : nullptr;
    *ctas = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (*ctas > 0) return cudaSuccess;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, fn, threads, 0);
    if (e == cudaSuccess && *ctas < 1) *ctas = 1;
    if (e == cudaSuccess && slot) slot->store(*ctas, std::memory_order_relaxed);
    return e;
  }
  cudaError_t allow(const void* fn, int bytes, int most) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && large[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && dev < kDevices) large[dev].store(true, std::memory_order_relaxed);
    return e;
  }
};

// Host checks shared by the operators' entry points.
inline bool known_type(int t) { return t == ZERO_FP16 || t == ZERO_BF16 || t == ZERO_FP32; }
inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace zero
