// Eviction by accumulated attention weight: for every request and KV head,
// choose the `keep` slots to keep of its n (the first S, the last R, and
// among the others those of the highest weight, ties to the lowest position)
// and move their K, V and weight rows, in order, to the front of the request's
// destination pages.
//
// Two kernels, chained by programmatic dependent launch:
//   * select, one block per (request, KV head): the k-th largest weight by a
//     radix search over order-preserving 32-bit keys (four histograms of eight
//     bits, from the top; the histogram of each holds the keys that share the
//     bits found so far), then one ordered pass that writes the positions of
//     the keys above it and of the first ones equal to it. No sort, no atomics
//     whose order could show: the histogram counts are sums, the positions come
//     from a prefix sum.
//   * move: each block takes a 64-byte column slice of K or of V of one
//     (request, KV head), or its weights, and walks the kept rows in order.
//     Kept positions ascend, so row j's source p_j >= j is never a
//     destination written before it: a tile of rows is read, the block meets
//     at a barrier, and the tile is written. That makes moving in place (the
//     destination table is the block table) safe with no copy in between,
//     since no two blocks share a byte.
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// Order-preserving key of a weight: larger weights have larger keys; NaN is
// below everything, -0 equals +0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_context(const EvictArgs& a, int b, bool record)
{
    int n = a.context_lens[b];
    const int cap = a.max_pages << a.ps_shift;
    if (n < 0 || n > cap) {
        if (record)
            atomicOr(a.err, PA_DEVERR_CONTEXT_LEN_BIT);
        n = n < 0 ? 0 : cap;
    }
    return n;
}

// Slot row of logical position pos of (table row bt, head h), or -1 for a page
// id outside the pool.
__device__ __forceinline__ int slot_row(const EvictArgs& a, const int32_t* bt, int h, int pos)
{
    const int phys = bt[pos >> a.ps_shift];
    if (unsigned(phys) >= unsigned(a.num_pages)) {
        atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
        return -1;
    }
    return ((phys * a.H_kv + h) << a.ps_shift) + (pos & ((1 << a.ps_shift) - 1));
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a)
{
    __shared__ int hist[256];
    __shared__ int found[2];                 // digit, keys above it within the prefix
    __shared__ int warp_sum[kSelWarps];      // keys above (low half) and equal (high half)
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.H_kv, h = blockIdx.x - b * a.H_kv;
    const int n = evict_context(a, b, tid == 0 && h == 0);
    int32_t* kept = a.kept + int64_t(blockIdx.x) * a.keep;
    const int len = n < a.keep ? n : a.keep;
    if (tid == 0 && h == 0)
        a.new_lens[b] = len;
    if (n <= a.keep) {
        for (int j = tid; j < a.keep; j += kSelThreads)
            kept[j] = j < n ? j : -1;
        return;
    }
    for (int j = tid; j < a.sinks; j += kSelThreads)
        kept[j] = j;
    for (int j = tid; j < a.recent; j += kSelThreads)
        kept[a.keep - a.recent + j] = n - a.recent + j;
    const int k = a.keep - a.sinks - a.recent;       // to choose among [lo, hi)
    if (k == 0)
        return;
    const int lo = a.sinks, hi = n - a.recent;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    auto key_at = [&](int pos) -> uint32_t {
        const int row = slot_row(a, bt, h, pos);
        return row < 0 ? 0u : weight_key(a.weight_pages[row]);
    };
    // The k-th largest key, eight bits at a time from the top.
    uint32_t prefix = 0;
    int want = k;                                    // rank among the keys that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256)
            hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int p = lo + tid; p < hi; p += kSelThreads) {
            const uint32_t key = key_at(p);
            if ((key & mask) == prefix)
                atomicAdd(&hist[(key >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // bins 255 - 8 lane down to 248 - 8 lane, counted from the top
            int c[8], sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                c[u] = hist[255 - 8 * lane - u];
                sum += c[u];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            int above = incl - sum;
            if (above < want && want <= incl) {
                int u = 0;
                while (above + c[u] < want)
                    above += c[u++];
                found[0] = 255 - 8 * lane - u;
                found[1] = above;
            }
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        want -= found[1];
        __syncthreads();
    }
    // prefix: the k-th largest key; `want` of the keys equal to it are kept.
    int above = 0, equal = 0;                        // before this round
    for (int p0 = lo; p0 < hi; p0 += kSelThreads) {
        const int p = p0 + tid;
        const uint32_t key = p < hi ? key_at(p) : 0u;
        const bool gt = p < hi && key > prefix, eq = p < hi && key == prefix;
        const uint32_t g = __ballot_sync(0xffffffffu, gt), e = __ballot_sync(0xffffffffu, eq);
        if (lane == 0)
            warp_sum[warp] = __popc(g) | (__popc(e) << 16);
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            before += w < warp ? warp_sum[w] : 0;
            all += warp_sum[w];
        }
        const uint32_t below = (1u << lane) - 1u;
        const int ga = above + (before & 0xffff) + __popc(g & below);
        const int ea = equal + (before >> 16) + __popc(e & below);
        if (gt || (eq && ea < want))
            kept[lo + ga + (ea < want ? ea : want)] = p;
        above += all & 0xffff;
        equal += all >> 16;
        __syncthreads();
    }
}

constexpr int kMoveThreads = 256;
constexpr int kSlice = 64;                   // bytes of a row per block
constexpr int kUnroll = 8;                   // rows in flight per thread

// T: uint4 with four threads per row slice, or float with one (the weights).
template <typename T, int kPerRow>
__device__ __forceinline__ void move_rows(const EvictArgs& a, T* pool, int64_t row_units, int unit,
                                          int b, int h, int len, const int32_t* kept)
{
    constexpr int kRows = kMoveThreads / kPerRow;
    constexpr int kTile = kRows * kUnroll;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int32_t* dt = a.dst_table + int64_t(b) * a.dst_max_pages;
    const int r0 = threadIdx.x / kPerRow;
    T* col = pool + unit;
    for (int j0 = 0; j0 < len; j0 += kTile) {
        T v[kUnroll];
        int dst[kUnroll];
        int src[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = j0 + u * kRows + r0;
            src[u] = j < len ? kept[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = j0 + u * kRows + r0;
            dst[u] = -1;
            if (src[u] >= 0) {
                src[u] = slot_row(a, bt, h, src[u]);
                dst[u] = slot_row(a, dt, h, j);
                if (src[u] < 0 || src[u] == dst[u])
                    dst[u] = -1;                     // bad page, or the row stays
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (dst[u] >= 0)
                v[u] = __ldcg(col + src[u] * row_units);
        __syncthreads();                             // the tile is read before any of it is written
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (dst[u] >= 0)
                __stcg(col + dst[u] * row_units, v[u]);
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = 2 * a.slices + 1;                // K slices, V slices, the weights
    const int64_t bh = blockIdx.x / per;
    const int part = int(blockIdx.x - bh * per);
    const int b = int(bh / a.H_kv), h = int(bh - int64_t(b) * a.H_kv);
    const int n = evict_context(a, b, false);
    const int len = n < a.keep ? n : a.keep;
    const int32_t* kept = a.kept + bh * a.keep;
    if (part == 2 * a.slices) {
        move_rows<float, 1>(a, a.weight_pages, 1, 0, b, h, len, kept);
    } else {
        const bool is_v = part >= a.slices;
        const int slice = part - (is_v ? a.slices : 0);
        move_rows<uint4, kSlice / 16>(a, reinterpret_cast<uint4*>(is_v ? a.value_pages : a.key_pages),
                                      a.row_bytes / 16,
                                      slice * (kSlice / 16) + int(threadIdx.x % (kSlice / 16)), b, h, len,
                                      kept);
    }
}

}  // namespace

cudaError_t launch_evict(EvictArgs a, cudaStream_t stream)
{
    a.slices = a.row_bytes / kSlice;
    const int64_t heads = int64_t(a.B) * a.H_kv;
    const int64_t moves = heads * (2 * a.slices + 1);
    if (moves >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(heads));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(unsigned(moves));
    cfg.blockDim = dim3(kMoveThreads);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace pa
