// The split of a decode call's work over blocks: the granules (runs of keys)
// of all segments (request, KV head, group of row tiles) form one stream, cut
// into equal contiguous ranges. Shared by the kernels that take such ranges.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ int clamp_context(int n, int cap, unsigned* err)
{
    if (n < 0 || n > cap) {
        atomicOr(err, PA_DEVERR_CONTEXT_LEN_BIT);
        n = n < 0 ? 0 : cap;
    }
    return n;
}

struct SegmentPos {
    int b, h, ms, seg;  // request, KV head, segment within the (b, h) rows
    int64_t seg_start;  // first granule of the segment in the stream
    int seg_len;        // granules in the segment
};

// The segment hm (0 <= hm < per_req) of request b. pre[b] = first granule of
// request b, gbr[b] = granules in each of its segments.
__device__ __forceinline__ SegmentPos segment_at(const int32_t* pre, const int32_t* gbr,
                                                 int per_req, int MS, int b, int hm)
{
    SegmentPos s;
    s.b = b;
    s.h = MS == 1 ? hm : hm / MS;
    s.ms = hm - s.h * MS;
    s.seg = b * per_req + hm;
    s.seg_len = gbr[b];
    s.seg_start = pre[b] + int64_t(hm) * s.seg_len;
    return s;
}

// The segment after s in the stream (segments are in (request, KV head, row
// tile group) order and none is empty).
__device__ __forceinline__ SegmentPos next_segment(const int32_t* pre, const int32_t* gbr,
                                                   int per_req, int MS, const SegmentPos& s)
{
    const int hm = s.seg - s.b * per_req + 1;
    return hm < per_req ? segment_at(pre, gbr, per_req, MS, s.b, hm)
                        : segment_at(pre, gbr, per_req, MS, s.b + 1, 0);
}

// Block index that processes the granule at unit position u.
__device__ __forceinline__ int64_t block_of_unit(int64_t u, int64_t units, int64_t grid)
{
    return udiv64((u + 1) * grid - 1, units);
}

// First granule whose unit position is >= u (the granule count if none),
// and the request b and segment hm within it that hold that granule (b = B
// if none), for the two unit positions u0 <= u1 at once (the two searches
// and their divisions interleave). Called by whole warps.
struct StreamPoint {
    int64_t x;
    int b, hm;
};
__device__ __forceinline__ void granules_at_units(const int32_t* pre, const int32_t* gbr, int B,
                                                  int per_req, int64_t u0, int64_t u1,
                                                  int64_t units, int pu, StreamPoint& p0,
                                                  StreamPoint& p1)
{
    const int lane = threadIdx.x & 31;
    const int64_t per_b = int64_t(pu) * per_req;
    auto pre_u = [&](int b) { return int64_t(pre[b]) + per_b * b; };
    // largest b with pre_u(b) <= u, for both u (pre_u(0) = 0 <= u); each
    // round samples 32 evenly spaced candidates of the remaining range, so
    // B <= 32 takes one round of one shared-memory read per lane
    int lo0 = 0, n0 = B, lo1 = 0, n1 = B;
    while (n0 > 32 || n1 > 32) {
        const int s0 = (n0 + 31) >> 5, s1 = (n1 + 31) >> 5;
        const bool ok0 = lane * s0 < n0 && pre_u(lo0 + lane * s0) <= u0;
        const bool ok1 = lane * s1 < n1 && pre_u(lo1 + lane * s1) <= u1;
        const int l0 = 31 - __clz(__ballot_sync(0xffffffffu, ok0));
        const int l1 = 31 - __clz(__ballot_sync(0xffffffffu, ok1));
        lo0 += l0 * s0;
        n0 = min(s0, n0 - l0 * s0);
        lo1 += l1 * s1;
        n1 = min(s1, n1 - l1 * s1);
    }
    const bool ok0 = lane < n0 && pre_u(lo0 + lane) <= u0;
    const bool ok1 = lane < n1 && pre_u(lo1 + lane) <= u1;
    lo0 += 31 - __clz(__ballot_sync(0xffffffffu, ok0));
    lo1 += 31 - __clz(__ballot_sync(0xffffffffu, ok1));
    auto finish = [&](int lo, int64_t u, StreamPoint& p) {
        if (u >= units) {
            p = StreamPoint{pre[B], B, 0};
            return;
        }
        const int gb = gbr[lo];
        const int64_t r = u - pre_u(lo);
        const int64_t hm = udiv64(r, gb + pu);
        const int64_t in = r - hm * (gb + pu) - pu;
        p = StreamPoint{pre[lo] + hm * gb + (in > 0 ? in : 0), lo, int(hm)};
    };
    finish(lo0, u0, p0);
    finish(lo1, u1, p1);
}

}  // namespace pa
