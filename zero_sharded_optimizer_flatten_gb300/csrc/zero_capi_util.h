// Status and error-message helpers shared by the C-ABI translation units.
#pragma once

#include <nvtx3/nvToolsExt.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>
#include <initializer_list>

#include "zero.h"

namespace zero {

// Thread-local message of the last failed call (see zero_last_error).
char* error_buffer();

// Launches issued since load (zero_launch_count).
extern std::atomic<int64_t> g_launches;

inline void clear_error() { error_buffer()[0] = '\0'; }

#if defined(__GNUC__)
__attribute__((format(printf, 2, 3)))
#endif
inline zero_status fail(zero_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(error_buffer(), 1024, fmt, ap);
  va_end(ap);
  return st;
}

// An NVTX range named after the C-ABI call, for timelines in Nsight tools
// (a no-op unless a tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// An argument's memory: rows of `width` bytes, `pitch` bytes apart.  p NULL, no
// rows or no width: none.
struct Extent {
  const char* name;
  const void* p;
  int64_t rows, pitch, width;
  const void* in_place = nullptr;  // an output: the input that it may be, row for row

  static Extent block(const char* name, const void* p, int64_t bytes, const void* in_place = nullptr) {
    return {name, p, 1, bytes, bytes, in_place};
  }
  bool overlaps(const Extent& out) const {  // out: one row
    if (!p || !out.p || rows < 1 || width < 1 || out.rows < 1 || out.width < 1) return false;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(out.p) - reinterpret_cast<uintptr_t>(p));
    if (at + out.width <= 0) return false;
    const int64_t r = at < width ? 0 : (at - width) / pitch + 1;  // the first row that ends past out's start
    return r < rows && r * pitch < at + out.width;
  }
  bool same_rows(const Extent& out) const {
    return p == out.p && (rows == 1 || pitch == width) && rows * width == out.width;
  }
};

// No output overlaps an input, but for the one that it may be in place of, or
// another output.
inline zero_status check_overlaps(const char* fn, std::initializer_list<Extent> outs,
                                  std::initializer_list<Extent> ins) {
  for (const Extent* o = outs.begin(); o != outs.end(); ++o) {
    for (const Extent& in : ins)
      if (in.overlaps(*o) && !(in.p == o->in_place && in.same_rows(*o)))
        return fail(ZERO_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, in.name);
    for (const Extent* m = outs.begin(); m != o; ++m)
      if (m->overlaps(*o)) return fail(ZERO_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, m->name);
  }
  return ZERO_OK;
}

}  // namespace zero
