// Plays two CTAs that copy through a ring of slots, announce and count bytes at
// the leading one's barriers (csrc/zero_drain.h), stopped at every combination
// of points, and checks that the waits afterwards end, and only when nothing is
// in flight any more.  Prints the number of endings.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "zero_drain.h"

using namespace zero;

namespace {

constexpr int kStages = 6;
constexpr int64_t kLeadBytes = 7, kOtherBytes = 5;  // of a copy

// A barrier of one arrival and counted bytes.
struct Bar {
  int64_t phase = 0, pending = 1, bytes = 0;
  void settle() {
    if (pending == 0 && bytes == 0) ++phase, pending = 1;
  }
  void announce(int64_t n) { bytes += n, --pending, settle(); }
  void count(int64_t n) { bytes -= n, settle(); }
  bool over(int64_t parity) const { return (phase & 1) != parity; }  // of the phase with that parity
};

// `done`: products over that many copies; lead, other: copies made; landed: how
// many of each have arrived (the rest are in flight).
bool ending(int64_t done, int64_t lead, int64_t other, int64_t lead_landed, int64_t other_landed) {
  std::vector<Bar> bars(kStages);
  for (int64_t j = 0; j < lead; ++j) {
    Bar& b = bars[j % kStages];
    b.announce(kLeadBytes + kOtherBytes);
    if (j < lead_landed) b.count(kLeadBytes);
    if (j < other_landed) b.count(kOtherBytes);
  }
  for (int64_t j = lead; j < other_landed; ++j) bars[j % kStages].count(kOtherBytes);
  for (int64_t j = 0; j < done; ++j)
    if (bars[j % kStages].phase <= j / kStages) return false;  // the play itself
  const Drain d(lead, other, kStages);
  if (d.last - d.first > kStages) return false;
  for (int64_t j = d.first; j < d.last; ++j) {
    Bar& b = bars[j % kStages];
    if (d.announce(j)) b.announce(kOtherBytes);
    else if (d.forgo(j)) b.count(kOtherBytes);
    const int64_t parity = (j / kStages) & 1;
    const bool lead_flies = j < lead && j >= lead_landed, other_flies = j < other && j >= other_landed;
    if ((lead_flies || other_flies) && b.over(parity)) return false;  // would not wait
    if (lead_flies) b.count(kLeadBytes);
    if (other_flies) b.count(kOtherBytes);
    if (!b.over(parity)) return false;  // would wait for ever
  }
  // nothing that flies was left out
  return d.first <= lead_landed || lead_landed >= lead ? d.first <= other_landed || other_landed >= other : false;
}

}  // namespace

int main() {
  long endings = 0;
  for (int64_t done = 0; done <= 3 * kStages; ++done)
    for (int64_t lead = done; lead <= done + kStages; ++lead)
      for (int64_t other = done; other <= done + kStages; ++other)
        for (int64_t a = done; a <= lead; ++a)
          for (int64_t b = done; b <= other; ++b, ++endings)
            if (!ending(done, lead, other, a, b)) {
              printf("done %ld, made %ld and %ld, landed %ld and %ld\n", long(done), long(lead), long(other), long(a), long(b));
              return 1;
            }
  printf("%ld\n", endings);
  return 0;
}
