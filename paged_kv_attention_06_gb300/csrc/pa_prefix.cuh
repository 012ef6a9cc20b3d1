// The prefixes that requests of a batch share: which one a request has, and its length.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ int prefix_len(const PrefixArgs& x, int p)
{
    const int n = __ldcg(x.lens + p);
    return n < 0 ? 0 : n > x.cap ? x.cap : n;
}

// The prefix of request b, starts[p] <= b < starts[p + 1], of `count` that start in
// ascending order (shared memory); -1 where it has none.
__device__ __forceinline__ int prefix_of(const int* starts, int count, int b)
{
    if (b < starts[0] || b >= starts[count])
        return -1;
    int lo = 0, hi = count;                // starts[lo] <= b < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= b)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The blocks of the few-row kernel behind a prefix that share units of work, two units a
// block at least.
__device__ __forceinline__ int64_t suffix_blocks(int64_t units, int grid)
{
    const int64_t most = (units + 1) / 2;
    return most < grid ? most : grid;
}

// Floats of a few-row state left as rows: O [8 NT][D], then (m, l) of each row.
__host__ __device__ constexpr int suffix_slot_floats(int D, int NT) { return 8 * NT * (D + 2); }

}  // namespace pa
