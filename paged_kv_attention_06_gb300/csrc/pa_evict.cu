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
#include <cooperative_groups.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

namespace cg = cooperative_groups;

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

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kFly = 8;                      // weights in flight per thread
// Keys that a block holds in shared memory after the one read of the weights;
// what lies behind them is read again in every pass.
constexpr int kSelKeys = 19 * 1024;
constexpr int kHistInts = 256 * 32;

// One cluster of `cluster_dim` blocks per (request, KV head), each with a run of the
// candidate positions. Histograms have a copy per lane, so that neither equal
// digits (most weights share a few exponents) nor banks collide: 32k keys took
// 45 us with one copy and one block.
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictArgs a, int cached)
{
    extern __shared__ uint32_t smem_keys[];  // [256][32] histogram copies, then [cached] keys
    __shared__ int sums[2][256];             // this block's histogram of a pass (by parity)
    __shared__ int counts[2];                // this block's keys above and equal
    __shared__ int found[3];                 // digit, keys above it within the prefix, keys of it
    __shared__ int2 warp_sum[kSelWarps];
    int* hist = reinterpret_cast<int*>(smem_keys);
    uint32_t* keys = smem_keys + kHistInts;
    grid_dependency_wait();
    grid_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x / C;
    const int b = bh / a.H_kv, h = bh - b * a.H_kv;
    const bool first = tid == 0 && h == 0 && rank == 0;
    const int n = evict_context(a, b, first);
    int32_t* kept = a.kept + int64_t(bh) * a.keep;
    if (first)
        a.new_lens[b] = n < a.keep ? n : a.keep;
    // All blocks of a cluster take the same way out, before any of them
    // reads another's shared memory.
    const int all = rank * kSelThreads + tid, step = C * kSelThreads;
    if (n <= a.keep) {
        for (int j = all; j < a.keep; j += step)
            kept[j] = j < n ? j : -1;
        return;
    }
    for (int j = all; j < a.sinks; j += step)
        kept[j] = j;
    for (int j = all; j < a.recent; j += step)
        kept[a.keep - a.recent + j] = n - a.recent + j;
    const int k = a.keep - a.sinks - a.recent;       // to choose among [sinks, n - recent)
    if (k == 0)
        return;
    const int total = n - a.recent - a.sinks;
    const int part = ((total + C - 1) / C + 31) & ~31;
    const int lo = a.sinks + rank * part;            // this block's candidates: [lo, lo + m)
    const int m = max(0, min(part, total - rank * part));
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    // The one read of the weights: kFly page ids, then kFly weights in flight.
    const int held = m < cached ? m : cached;
    for (int p0 = tid; p0 < held; p0 += kSelThreads * kFly) {
        int row[kFly];
        float w[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const int p = p0 + u * kSelThreads;
            row[u] = p < held ? slot_row(a, bt, h, lo + p) : -1;
        }
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            w[u] = row[u] >= 0 ? a.weight_pages[row[u]] : NAN;
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            if (p0 + u * kSelThreads < held)
                keys[p0 + u * kSelThreads] = weight_key(w[u]);
    }
    auto key_at = [&](int p) -> uint32_t {
        if (p < held)
            return keys[p];
        const int row = slot_row(a, bt, h, lo + p);
        return row < 0 ? 0u : weight_key(a.weight_pages[row]);
    };

    // The k-th largest key, eight bits at a time from the top; done as soon as
    // all keys that share the bits found are wanted.
    uint32_t prefix = 0;
    int want = k;                                    // rank among the keys that share the prefix
    bool all_equal = false;
    for (int shift = 24; shift >= 0 && !all_equal; shift -= 8) {
        const int buf = (shift >> 3) & 1;
        for (int i = tid; i < kHistInts; i += kSelThreads)
            hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int p = tid; p < m; p += kSelThreads) {
            const uint32_t key = key_at(p);
            if ((key & mask) == prefix)
                atomicAdd(&hist[((key >> shift) & 255u) * 32 + lane], 1);
        }
        __syncthreads();
        {
            // two threads a bin, each half of the copies, rotated over the banks
            const int bin = tid >> 1;
            int c = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                c += hist[bin * 32 + (tid & 1) * 16 + ((i + bin) & 15)];
            c += __shfl_xor_sync(0xffffffffu, c, 1);
            if ((tid & 1) == 0)
                sums[buf][bin] = c;
        }
        cluster.sync();
        if (warp == 0) {
            // bins 255 - 8 lane down to 248 - 8 lane, counted from the top
            int c[8], sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                c[u] = 0;
            for (int r = 0; r < C; ++r) {
                const int* from = cluster.map_shared_rank(&sums[buf][0], r);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    c[u] += from[255 - 8 * lane - u];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                sum += c[u];
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            int above = incl - sum;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (above < want && want <= above + c[u]) {
                    found[0] = 255 - 8 * lane - u;
                    found[1] = above;
                    found[2] = c[u];
                }
                above += c[u];
            }
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        want -= found[1];
        all_equal = want == found[2];
    }
    // Kept: the keys above prefix, and the first `want` of those equal to it;
    // where all that share the found bits are wanted, the keys from prefix up.
    // Each warp takes a run of positions: counts first, then the places.
    const int run = ((m + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int r0 = warp * run, r1 = min(m, r0 + run);
    auto judge = [&](int p, uint32_t* g, uint32_t* e, bool* gg, bool* ee) {
        const uint32_t key = p < r1 ? key_at(p) : 0u;
        *gg = p < r1 && (all_equal ? key >= prefix : key > prefix);
        *ee = p < r1 && !all_equal && key == prefix;
        *g = __ballot_sync(0xffffffffu, *gg);
        *e = __ballot_sync(0xffffffffu, *ee);
    };
    uint32_t g, e;
    bool gg, ee;
    int gt = 0, eq = 0;
    for (int p0 = r0; p0 < r1; p0 += 32) {
        judge(p0 + lane, &g, &e, &gg, &ee);
        gt += __popc(g);
        eq += __popc(e);
    }
    if (lane == 0)
        warp_sum[warp] = make_int2(gt, eq);
    __syncthreads();
    int above = 0, equal = 0;                        // kept-above and equal keys before this warp's
    for (int w = 0; w < warp; ++w) {
        above += warp_sum[w].x;
        equal += warp_sum[w].y;
    }
    if (warp == kSelWarps - 1 && lane == 0) {
        counts[0] = above + gt;
        counts[1] = equal + eq;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
        const int* from = cluster.map_shared_rank(&counts[0], r);
        above += from[0];
        equal += from[1];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int p0 = r0; p0 < r1; p0 += 32) {
        judge(p0 + lane, &g, &e, &gg, &ee);
        const int ga = above + __popc(g & below);
        const int ea = equal + __popc(e & below);
        if (gg || (ee && ea < want))
            kept[a.sinks + ga + (ea < want ? ea : want)] = lo + p0 + lane;
        above += __popc(g);
        equal += __popc(e);
    }
    cluster.sync();                                  // no block ends while another reads its counts
}

constexpr int kMoveThreads = 256;
constexpr int kSlice = 64;                   // bytes of a row per block
constexpr int kUnroll = 4;                   // rows of a tile per thread
constexpr int kChunkRows = 2048;             // rows per block where order does not matter
constexpr int kTableInts = 6 * 1024;         // page ids staged in shared memory

// Rows [j_begin, j_end) of the kept ones. T: uint4 with four threads per row
// slice, or float with one (the weights). bt, dt: the request's page ids
// (shared memory, or global where they are many). One tile is in registers
// while the next one's rows are read: a row's source is never a destination of
// an earlier tile, so reading ahead is safe; the barrier keeps a tile's writes
// behind every thread's reads of it.
template <typename T, int kPerRow>
__device__ __forceinline__ void move_rows(const EvictArgs& a, T* pool, int64_t row_units, int unit,
                                          const int32_t* bt, const int32_t* dt, int h, int j_begin,
                                          int j_end, const int32_t* kept)
{
    constexpr int kRows = kMoveThreads / kPerRow;
    constexpr int kTile = kRows * kUnroll;
    const int r0 = threadIdx.x / kPerRow;
    T* col = pool + unit;
    int pos[kUnroll];                        // kept positions of the tile to be read next
    T v[2][kUnroll];
    uint32_t moves[2];                       // bit u: row u of the tile in v goes somewhere
    auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = j0 + u * kRows + r0;
            pos[u] = j < j_end ? kept[j] : -1;
        }
    };
    auto read = [&](int j0, int k) {
        moves[k] = 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (pos[u] >= 0) {
                const int src = slot_row(a, bt, h, pos[u]);
                const int dst = slot_row(a, dt, h, j0 + u * kRows + r0);
                if (src >= 0 && dst >= 0 && src != dst) {   // else a bad page, or the row stays
                    moves[k] |= 1u << u;
                    v[k][u] = __ldcg(col + src * row_units);
                }
            }
    };
    auto write = [&](int j0, int k) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (moves[k] >> u & 1u)
                __stcg(col + slot_row(a, dt, h, j0 + u * kRows + r0) * row_units, v[k][u]);
    };
    fetch(j_begin);
    read(j_begin, 0);
    fetch(j_begin + kTile);
    for (int j0 = j_begin; j0 < j_end; j0 += 2 * kTile) {
        read(j0 + kTile, 1);
        fetch(j0 + 2 * kTile);
        __syncthreads();
        write(j0, 0);
        read(j0 + 2 * kTile, 0);
        fetch(j0 + 3 * kTile);
        __syncthreads();
        write(j0 + kTile, 1);
    }
}

__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictArgs a)
{
    __shared__ int32_t table[kTableInts];
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = 2 * a.slices + 1;                // K slices, V slices, the weights
    int64_t blk = blockIdx.x;
    const int part = int(blk % per);
    blk /= per;
    const int chunk = int(blk % a.chunks);
    const int64_t bh = blk / a.chunks;
    const int b = int(bh / a.H_kv), h = int(bh - int64_t(b) * a.H_kv);
    const int n = evict_context(a, b, false);
    const int len = n < a.keep ? n : a.keep;
    const int32_t* kept = a.kept + bh * a.keep;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int32_t* dt = a.dst_table + int64_t(b) * a.dst_max_pages;
    const int dst_ids = (len + (1 << a.ps_shift) - 1) >> a.ps_shift;
    // Chunks of rows in any order where no destination page is one of the
    // request's own; otherwise its rows in order, in the first chunk's block.
    int j_begin = chunk * kChunkRows, j_end = min(len, j_begin + kChunkRows);
    if (a.chunks > 1) {
        int own = 0;
        for (int i = threadIdx.x; i < dst_ids; i += kMoveThreads)
            own |= dt[i] == bt[i];
        if (__syncthreads_or(own)) {
            if (chunk > 0)
                return;
            j_end = len;
        }
    } else {
        j_end = len;
    }
    if (j_begin >= j_end)
        return;
    // The page ids that these rows need.
    const int s0 = kept[j_begin] >> a.ps_shift, s1 = kept[j_end - 1] >> a.ps_shift;
    const int d0 = j_begin >> a.ps_shift, d1 = (j_end - 1) >> a.ps_shift;
    const int ns = s1 - s0 + 1, nd = d1 - d0 + 1;
    if (ns + nd <= kTableInts) {
        for (int i = threadIdx.x; i < ns; i += kMoveThreads)
            table[i] = bt[s0 + i];
        for (int i = threadIdx.x; i < nd; i += kMoveThreads)
            table[ns + i] = dt[d0 + i];
        bt = table - s0;
        dt = table + ns - d0;
        __syncthreads();
    }
    if (part == 2 * a.slices) {
        move_rows<float, 1>(a, a.weight_pages, 1, 0, bt, dt, h, j_begin, j_end, kept);
    } else {
        const bool is_v = part >= a.slices;
        const int slice = part - (is_v ? a.slices : 0);
        move_rows<uint4, kSlice / 16>(a, reinterpret_cast<uint4*>(is_v ? a.value_pages : a.key_pages),
                                      a.row_bytes / 16,
                                      slice * (kSlice / 16) + int(threadIdx.x % (kSlice / 16)), bt, dt, h,
                                      j_begin, j_end, kept);
    }
}

}  // namespace

cudaError_t launch_evict(EvictArgs a, int device, int sm_count, cudaStream_t stream)
{
    a.slices = a.row_bytes / kSlice;
    const int64_t heads = int64_t(a.B) * a.H_kv;
    const int64_t cap = int64_t(a.max_pages) << a.ps_shift;
    const int64_t rows = cap < a.keep ? cap : a.keep;
    a.chunks = a.dst_table == a.block_table ? 1 : int((rows + kChunkRows - 1) / kChunkRows);
    const int64_t moves = heads * (2 * a.slices + 1) * a.chunks;
    // Blocks per (request, KV head) for the choice: more while the GPU has room
    // for them (two per SM) and each still has a few keys per thread.
    int C = 1;
    while (C < kMaxCluster && heads * C * 2 <= 2 * int64_t(sm_count) && cap > 4 * kSelThreads * C)
        C *= 2;
    if (moves >= (int64_t(1) << 31) || heads * C >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    const int64_t share = (cap + C - 1) / C + 31;
    const int cached = int(share < kSelKeys ? share : kSelKeys);
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev];
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    cudaError_t e;
    if (!raised[device].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (kHistInts + kSelKeys) * int(sizeof(uint32_t)));
        if (e != cudaSuccess)
            return e;
        raised[device].store(true, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(C);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(heads * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = size_t(kHistInts + cached) * sizeof(uint32_t);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cached);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(unsigned(moves));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace pa
