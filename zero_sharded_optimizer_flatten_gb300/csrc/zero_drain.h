// Which copies a pair of CTAs may leave in flight when one of its waits has
// given up, and what their barriers still lack. Index arithmetic only, for the
// host compiler as well.
#pragma once

#include <stdint.h>

#include "zero_pieces.h"

namespace zero {

// Copy j of each CTA goes to slot j % stages of its own memory; both count at the
// leading CTA's barrier of that slot, whose phase j / stages ends when the leading
// CTA has announced the bytes of both and these have arrived. A copy is made once
// the products have read the slot's one before, so only the last `stages` of the
// CTA that is ahead can be in flight, and neither is more than `stages` ahead.
struct Drain {
  int64_t lead, other;  // copies that the leading CTA announced and made, that the other one made
  int64_t first, last;  // the copies to wait for
  ZERO_HD Drain(int64_t lead_, int64_t other_, int stages) : lead(lead_), other(other_) {
    last = lead > other ? lead : other;
    first = last > stages ? last - stages : 0;
  }
  // The other CTA's bytes of copy j were not announced, or will not come.
  ZERO_HD bool announce(int64_t j) const { return j >= lead; }
  ZERO_HD bool forgo(int64_t j) const { return j >= other; }
};

}  // namespace zero
