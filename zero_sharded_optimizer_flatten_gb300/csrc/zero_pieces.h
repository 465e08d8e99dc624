// How a row of elements of any length and start falls into 16-byte pieces, and
// which bytes a piece's read touches where it starts off the boundaries.
// Address arithmetic only, for the host compiler as well.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define ZERO_HD __host__ __device__ __forceinline__
#else
#define ZERO_HD inline
#endif

namespace zero {

// A row that is written, `elem` bytes an element: `head` single columns up to
// the first 16-byte boundary, `pieces`, and single columns again, `ends` of
// them in all.  drop_first, drop_last: single columns in place of these pieces.
struct RowPieces {
  int cols;  // of a piece
  int head, pieces, ends;
  ZERO_HD RowPieces(uintptr_t row, int hidden, int elem, bool drop_first, bool drop_last) : cols(16 / elem) {
    const int to_boundary = static_cast<int>((0 - row) & 15) / elem;
    head = to_boundary < hidden ? to_boundary : hidden;
    pieces = (hidden - head) / cols;
    if (drop_first || drop_last) {
      if (drop_first) head += pieces > 0 ? cols : 0;
      pieces -= static_cast<int>(drop_first) + static_cast<int>(drop_last);
      if (pieces < 0) pieces = 0;
    }
    ends = hidden - pieces * cols;
  }
  ZERO_HD int column(int piece) const { return head + piece * cols; }
  ZERO_HD int end_column(int e) const { return e < head ? e : e + pieces * cols; }
};

// A window: 16 bytes that start `shift` bytes after a boundary, read as the one
// or two aligned pieces that hold them: 16 bytes from the boundary and 16 from
// this many bytes after it.
ZERO_HD int window_second(int shift) { return shift ? 16 : 0; }

// Whether the window of a row's last piece reaches past the row's end: the
// low bits of the ends of the row that is read and of the one that is written
// (whose last piece ends on a boundary).
ZERO_HD bool window_passes(uint32_t read_end, uint32_t written_end) {
  const uint32_t tail = written_end & 15u;
  return ((read_end - tail) & 15u) - 1u < 15u - tail;
}

}  // namespace zero
