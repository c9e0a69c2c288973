// joinflag.h -- the two sides of a join's flag in global memory (grouped.cu).
//
// A flag belongs to the worker that hands partial sums over and to the one that
// takes them in.  The first sets it to the launch's epoch; the second waits for
// that value and sets the flag back to 0.  A side whose wait has run out (here or
// anywhere else in its CTA) still visits the flag, once, and leaves the mark of
// having given up; whichever side comes second sets the flag back to 0.  So a
// launch that has ended leaves no flag behind, whatever happened in it: a captured
// launch has the same epoch on every replay, and would take a flag that an
// abandoned one left for its own.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define RNL_HOST_DEVICE __host__ __device__
#else
#define RNL_HOST_DEVICE
#endif

namespace rnl {

// What a side that gives up leaves in the flag.
RNL_HOST_DEVICE inline uint64_t join_gave_up(uint64_t epoch) { return ~epoch; }

// What a visit found in the flag: whether the other side has been there in this launch.
RNL_HOST_DEVICE inline bool join_is_second(uint64_t found, uint64_t epoch) {
  return found == epoch || found == join_gave_up(epoch);
}

}  // namespace rnl
