// Where packed sequences' offsets lead: plain integer arithmetic (no HIP), so that the host
// tests can compile it on its own.  Nothing is assumed of the offsets: what comes out is a
// sequence of the call, a row of its arrays or an input of a state.
#pragma once

#include <cstdint>

namespace sla {

// The sequence of step t: the last one that begins at t or before (the first if
// none does), so a valid index whatever the offsets hold.
__device__ __forceinline__ int64_t sequence_of(const int64_t* offsets, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// An offset as a row, not before `least` (0 <= least <= steps).
__device__ __forceinline__ int64_t row_at(int64_t offset, int64_t least, int64_t steps) {
  const int64_t row = offset < least ? least : offset;
  return row < steps ? row : steps;
}

// Which of a state's `taps` - 1 inputs stands for time t of a sequence that begins at
// `begin` (t < begin).
__device__ __forceinline__ int64_t state_at(int64_t t, int64_t begin, int64_t taps) {
  const int64_t j = (int64_t)((uint64_t)t - (uint64_t)begin) + taps - 1;
  return j < 0 ? 0 : j < taps - 2 ? j : taps - 2;
}

}  // namespace sla
