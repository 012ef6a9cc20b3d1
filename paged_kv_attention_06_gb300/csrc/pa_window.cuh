// The keys that a prefill's item (128 query rows of a request) visits under a
// sliding window, as the tiles of the prefill kernels take them.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// The keys of an item with a sliding window: those of [0, sinks), rounded up to
// whole boxes (`sink_keys`), then those from `start` on, the first key that the
// item's first row sees through the window rounded down to a box; one run
// from 0 where the two would meet. Boxes lie within a page and none is touched
// that no row sees. The two runs are laid end to end and cut into tiles of 128
// places, so the sinks rarely cost a tile of their own: key j is place j before
// sink_keys and place j + shift from there on.
struct WindowSpan {
    int sink_keys, start, shift;
    int first_seen;      // place of the first key that a row sees through the window
};
template <typename Args>
__device__ __forceinline__ WindowSpan window_span(const Args& a, int n, int row0)
{
    WindowSpan s;
    const int first = int(max(int64_t(0), int64_t(n) - a.L + row0 - a.window + 1));
    const int start = first & ~(a.box_rows - 1);
    const bool apart = start > a.sinks;
    s.sink_keys = apart ? (a.sinks + a.box_rows - 1) & ~(a.box_rows - 1) : 0;
    s.start = apart ? start : 0;
    s.shift = s.sink_keys - s.start;
    s.first_seen = first + s.shift;
    return s;
}

}  // namespace pa
