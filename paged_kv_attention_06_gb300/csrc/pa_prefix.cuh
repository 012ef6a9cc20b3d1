// The prefixes that requests of a batch share: which one a request has, and its length.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Prefix p belongs to the requests starts[p] .. starts[p + 1] - 1. Where the starts do
// not ascend within the batch (PA_DEVERR_PREFIX), each is taken as the largest so
// far, so that both kernels see the same division.
__device__ __forceinline__ int prefix_start(const PrefixArgs& x, int p, int B)
{
    const int s = __ldg(x.starts + p);
    return s < 0 ? 0 : s > B ? B : s;
}

__device__ __forceinline__ int prefix_len(const PrefixArgs& x, int p)
{
    const int n = __ldg(x.lens + p);
    return n < 0 ? 0 : n > x.cap ? x.cap : n;
}

// Tokens of request b's prefix; 0 where it has none.
__device__ __forceinline__ int prefix_of(const PrefixArgs& x, int b)
{
    if (x.count == 0 || b < __ldg(x.starts) || b >= __ldg(x.starts + x.count))
        return 0;
    int lo = 0, hi = x.count;              // starts[lo] <= b < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(x.starts + mid) <= b)
            lo = mid;
        else
            hi = mid;
    }
    return prefix_len(x, lo);
}

// Floats of a few-row state left as rows: O [8 NT][D], then (m, l) of each row.
__host__ __device__ constexpr int suffix_slot_floats(int D, int NT) { return 8 * NT * (D + 2); }

}  // namespace pa
