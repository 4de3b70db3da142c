// qmx_ring.h -- what a wave of k_mx_tile may still have on the way when it goes on to the next chunk.
//
// Memory operations of a wave complete in the order in which they were issued, and a
// wait leaves the last N of them on the way.  Chunk c is issued at step c - stages
// (the first `stages` in front of the loop) by `copies` operations; step 4 q issues the exponents of the next
// quad as well, where there is one to come.  Step c waits for chunk c + 1.
#pragma once

namespace qmx_ring {

// N of step c = 4 q + j.  exponents: as many operations as step 4 q has issued for them, and that must be none where nothing
// uses them, since the compiler then leaves them out.  Those issued in a later step than chunk c + 1 may be on the way
// too; in the same step, j == stages - 1, the order is the compiler's.
constexpr int may_be_on_the_way(int stages, int copies, int exponents, int j) {
  return (stages - 2) * copies + (j >= 1 && j < stages - 1 ? exponents : 0);
}

}  // namespace qmx_ring
