// segments.hpp -- where a packed batch's rows belong: segment i is rows starts[i] to
// starts[i + 1] - 1, the offsets in device memory (a captured graph replays with others).
#pragma once

#include "common.hpp"

namespace svdq {

// The last of n segments (n >= 1) whose first row is at or before `row`, or -1: the segment that
// holds the row if any does, where the offsets do not decrease (empty ones among equal offsets are
// never the last).  Each step tries 64 offsets, one a lane; every lane of the wave calls it and
// gets the same answer, which lies in [-1, n) for any offsets.
__device__ __forceinline__ int find_segment(const int* starts, int n, int row) {
    const int lane = threadIdx.x & 63;
    int lo = 0, len = n;   // the candidates
    while (true) {
        const int step = (len + 63) >> 6, i = lo + lane * step;
        const int before = __popcll(__ballot(lane * step < len && starts[min(i, n - 1)] <= row));
        if (before == 0) return lo - 1;   // only in the first step where the offsets do not decrease
        const int at = lo + (before - 1) * step;
        if (step == 1) return at;
        len = min(step, lo + len - at);
        lo = at;
    }
}

}  // namespace svdq
