// rr_search.h -- one round of a warp's common search in a sorted list: plain
// arithmetic, so that the host can follow a search step by step too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define RR_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RR_HOST_DEVICE inline
#endif

namespace rr {

// The warp looks for a window of values in the sorted list's range [lo, hi):
// its 32 lanes sample every search_step(lo, hi)-th key.
RR_HOST_DEVICE uint32_t search_step(uint32_t lo, uint32_t hi) { return (hi - lo + 31) / 32; }

// The narrower range after a round in which `below` samples were below the
// window and `within` were not above it (below <= within: the list is sorted).
// False where the round did not halve the range.  So it goes where one value's
// run fills the range: its ends then move by a sample or by a single key a
// round, and a binary search by every lane for itself is shorter.
RR_HOST_DEVICE bool search_narrow(uint32_t& lo, uint32_t& hi, uint32_t below, uint32_t within)
{
    const uint32_t step = search_step(lo, hi), size = hi - lo;
    const uint32_t from = below ? lo + (below - 1) * step + 1 : lo;
    if (within * (uint64_t)step < size) hi = lo + within * step;
    lo = from;
    return hi - lo <= size / 2;
}

}  // namespace rr
