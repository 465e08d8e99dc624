// Rows that start anywhere or end inside 16 bytes, by the 16-byte pieces of the
// row that is written.
#pragma once

#include "zero_pieces.h"
#include "zero_rows.cuh"

namespace zero {

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

}  // namespace zero
