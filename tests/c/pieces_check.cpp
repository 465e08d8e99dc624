// Walks every window that the row kernels read for rows of any length and
// start (csrc/zero_pieces.h) and checks that it lies in the rows that exist,
// and that each column is taken once.  Prints the number of windows.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "zero_pieces.h"

using namespace zero;

namespace {

long windows = 0;

// Row `row` of an array of H-element rows that starts at `in`, of which `kept`
// have to exist, read by the pieces of a row at `out`: single columns at the
// first row's start (`more`: of any row), and where a window would pass its
// row's end (of any row).
bool read_row(uintptr_t out, uintptr_t in, int64_t row, int64_t kept, int H, int elem, bool more) {
  const uintptr_t at = in + row * H * elem, row_end = at + H * elem, end = in + kept * H * elem;
  const bool passes = window_passes(static_cast<uint32_t>(row_end), static_cast<uint32_t>(out + H * elem));
  const bool first = row == 0 || more, last = passes || more;
  const RowPieces f(out, H, elem, first, last);
  std::vector<int> taken(H, 0);
  for (int u = 0; u < f.pieces; ++u) {
    const int c = f.column(u);
    const uintptr_t p = at + static_cast<uintptr_t>(c) * elem;
    const int shift = static_cast<int>(p & 15);
    const uintptr_t touched = p - shift, last_touched = touched + window_second(shift);
    ++windows;
    if ((out + static_cast<uintptr_t>(c) * elem) % 16 != 0 || last_touched % 16 != 0) return false;
    if (touched < in || last_touched + 16 > end || last_touched + 16 < p + 16) return false;
    if (shift && last_touched + 16 > row_end) return false;  // not even the next row
    for (int k = 0; k < f.cols; ++k) ++taken[c + k];
  }
  for (int e = 0; e < f.ends; ++e) {
    const int c = f.end_column(e);
    if (c < 0 || c >= H) return false;
    ++taken[c];
  }
  for (int c = 0; c < H; ++c)
    if (taken[c] != 1) return false;
  return true;
}

}  // namespace

int main() {
  const uintptr_t base = uintptr_t(1) << 40;
  for (int elem = 2; elem <= 4; elem += 2)
    for (int H = 1; H <= 70; ++H)
      for (int out = 0; out < 16; out += elem)
        for (int in = 0; in < 16; in += elem)
          for (int64_t kept = 1; kept <= 9; ++kept)
            for (int64_t row = 0; row < kept; ++row)
              for (int more = 0; more < 2; ++more)
                if (!read_row(base + out, 2 * base + in, row, kept, H, elem, more)) {
                  printf("elem %d H %d out %d in %d row %ld of %ld more %d\n", elem, H, out, in, (long)row,
                         (long)kept, more);
                  return 1;
                }
  printf("%ld\n", windows);
  return 0;
}
