// Eviction by accumulated attention weight: for every request and KV head,
// choose the `keep` slots to keep of its n (the first S, the last R, and
// among the others those of the highest weight, ties to the lowest position)
// and move their K, V and weight rows, in order, to the front of the request's
// destination pages.
//
// Two kernels, chained by programmatic dependent launch:
//   * select, a cluster of 1 to 8 blocks per (request, KV head): the k-th
//     largest weight by a radix search over order-preserving 32-bit keys (histograms of 11, 11 and
//     10 bits, from the top; each counts the keys that share the bits found so
//     far), then one ordered pass that writes the positions of
//     the keys above it and of the first ones equal to it. No sort, no atomics
//     whose order could show: the histogram counts are sums, the positions come
//     from a prefix sum.
//   * move: each block takes rows of K or of V of one (request, KV head), or its
//     weights. In place (the destination table is the block table) a block takes
//     a 64-byte column slice and walks all kept rows in order: kept positions
//     ascend, so row j's source p_j >= j is never a destination written before
//     it; a tile of rows is read, the block meets at a barrier, and the tile is
//     written. No copy in between, since no two blocks share a byte. Into other
//     pages the order is free, and a block takes whole rows of a part of them.
//
// The move is bound by memory (each kept row read and written once), the choice
// by the latency of its passes. Measured (one call of a replayed graph): 8
// requests of 16k-32k tokens to 8192 per head, 549 MB, 114 us (131 in place; e4m3 pools,
// 281 MB, 73 and 108); with 16 rows kept, nearly the choice alone, 23 us; one request of
// 1280 to 1024, 8.6.
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
constexpr int kFly = 8;                      // keys of a batch per thread
constexpr int kBatch = kSelThreads * kFly;
// Keys that a block holds in shared memory after the one read of the weights;
// what lies behind them is read again in every pass.
constexpr int kSelKeys = 4 * kBatch;
// Digits of a key, from the top: shift and bins. The first holds the sign, the
// exponent and two bits of the mantissa, so that weights of like size spread
// over bins; after it few keys are left to count.
constexpr int kPasses = 3;
__host__ __device__ constexpr int digit_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__host__ __device__ constexpr int digit_bins(int pass) { return pass == 2 ? 1024 : 2048; }
__host__ __device__ constexpr int digit_offset(int pass) { return 2048 * pass; }
constexpr int kBins = 2048 + 2048 + 1024;

// One cluster of C blocks per (request, KV head), each with a run of the
// candidate positions and a histogram of its own. A block adds its bins that
// are not empty (few) to the totals of every block of the cluster, so after one
// cluster barrier a pass each block scans the totals itself; reading the
// others' histograms instead took 12 us in the first pass at C = 8.
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictArgs a, int cached)
{
    extern __shared__ uint32_t smem_keys[];  // own bins, totals, then [cached] keys
    __shared__ int2 before[kMaxCluster];     // keys above and equal in each block of the cluster
    __shared__ int found[3];                 // digit, keys above it within the prefix, keys of it
    __shared__ int scan[kSelWarps];
    __shared__ alignas(16) int tally[kFly * kSelWarps];   // above | equal << 16, by (u, warp)
    __shared__ int2 mine;                    // this block's keys above and equal
    int* own = reinterpret_cast<int*>(smem_keys);
    int* totals = own + kBins;
    uint32_t* keys = smem_keys + 2 * kBins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 2 * kBins / 4; i += kSelThreads)
        reinterpret_cast<int4*>(own)[i] = make_int4(0, 0, 0, 0);
    if (tid == 0)
        mine = make_int2(0, 0);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    // The totals are clear in every block: waited for before the first addition.
    if (C > 1)
        cluster.barrier_arrive();
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int bh = blockIdx.x / C;
    const int b = bh / a.H_kv, h = bh - b * a.H_kv;
    const bool first = tid == 0 && h == 0 && rank == 0;
    const int n = evict_context(a, b, first);
    int32_t* kept = a.kept + int64_t(bh) * a.keep;
    if (first)
        a.new_lens[b] = n < a.keep ? n : a.keep;
    const int all = rank * kSelThreads + tid, step = C * kSelThreads;
    const int k = a.keep - a.sinks - a.recent;       // to choose among [sinks, n - recent)
    if (n <= a.keep) {
        for (int j = all; j < a.keep; j += step)
            kept[j] = j < n ? j : -1;
    } else {
        for (int j = all; j < a.sinks; j += step)
            kept[j] = j;
        for (int j = all; j < a.recent; j += step)
            kept[a.keep - a.recent + j] = n - a.recent + j;
    }
    if (n <= a.keep || k == 0) {                     // the same in every block of the cluster
        if (C > 1)
            cluster.barrier_wait();
        return;
    }
    const int total = n - a.recent - a.sinks;
    const int part = ((total + C - 1) / C + 31) & ~31;
    const int lo = a.sinks + rank * part;            // this block's candidates: [lo, lo + m)
    const int m = max(0, min(part, total - rank * part));
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    // A batch of keys: thread tid holds positions q0 + u * kSelThreads + tid. From
    // memory, the page ids are in flight together, then the weights.
    auto read_batch = [&](int q0, uint32_t* key) {
        int row[kFly];
        float w[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const int p = q0 + u * kSelThreads + tid;
            row[u] = p < m ? slot_row(a, bt, h, lo + p) : -1;
        }
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            w[u] = row[u] >= 0 ? a.weight_pages[row[u]] : NAN;
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            key[u] = weight_key(w[u]);
    };
    auto batch = [&](int q0, uint32_t* key) {
        if (q0 + kBatch <= cached) {
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                key[u] = keys[q0 + u * kSelThreads + tid];
        } else {
            read_batch(q0, key);
        }
    };
    auto live = [&](int q0, int u) { return q0 + u * kSelThreads + tid < m; };
    // A key into a histogram; a warp whose keys share the digit adds once.
    auto count = [&](int* to, int digit, bool counts) {
        const unsigned who = __ballot_sync(0xffffffffu, counts);
        if (who == 0)
            return;
        const int lead = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !counts || digit == lead)) {
            if (lane == __ffs(who) - 1)
                atomicAdd(&to[lead], __popc(who));
        } else if (counts) {
            atomicAdd(&to[digit], 1);
        }
    };

    // The k-th largest key, from the top digit down; done as soon as all keys
    // that share the bits found are wanted.
    uint32_t prefix = 0;
    int want = k;                                    // rank among the keys that share the prefix
    bool all_equal = false;
#pragma unroll 1
    for (int pass = 0; pass < kPasses && !all_equal; ++pass) {
        const int shift = digit_shift(pass), bins = digit_bins(pass);
        int* bin = own + digit_offset(pass);
        int* tot = totals + digit_offset(pass);
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << digit_shift(pass - 1);
        for (int q0 = 0; q0 < m; q0 += kBatch) {
            uint32_t key[kFly];
            if (pass == 0) {                         // the one read of the weights
                read_batch(q0, key);
                if (q0 + kBatch <= cached) {
#pragma unroll
                    for (int u = 0; u < kFly; ++u)
                        keys[q0 + u * kSelThreads + tid] = key[u];
                }
            } else {
                batch(q0, key);
            }
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                if (q0 + u * kSelThreads < m)
                    count(bin, int(key[u] >> shift) & (bins - 1), live(q0, u) && (key[u] & mask) == prefix);
        }
        __syncthreads();
        const int* sum_of = bin;
        if (C > 1) {
            if (pass == 0)
                cluster.barrier_wait();              // every block's totals are clear
            for (int i = tid; i < bins; i += kSelThreads) {
                const int c = bin[i];
                if (c != 0)
                    for (int r = 0; r < C; ++r)
                        atomicAdd(cluster.map_shared_rank(tot, r) + i, c);
            }
            cluster.sync();
            sum_of = tot;
        }
        // Bins from the top, four a thread (in the last pass the upper half of
        // the threads has none).
        const int base = bins - 4 * (tid + 1);
        int4 c = make_int4(0, 0, 0, 0);
        if (base >= 0)
            c = *reinterpret_cast<const int4*>(sum_of + base);
        const int sum = c.x + c.y + c.z + c.w;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int above = incl - sum;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w)
            above += w < warp ? scan[w] : 0;
        const int each[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (above < want && want <= above + each[u]) {
                found[0] = base + 3 - u;
                found[1] = above;
                found[2] = each[u];
            }
            above += each[u];
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        want -= found[1];
        all_equal = want == found[2];
    }
    // Kept: the keys above prefix, and the first `want` of those equal to it;
    // where all that share the found bits are wanted, the keys from prefix up.
    auto above_it = [&](uint32_t key) { return all_equal ? key >= prefix : key > prefix; };
    auto equal_it = [&](uint32_t key) { return !all_equal && key == prefix; };
    int above = 0, equal = 0;                        // in the blocks and batches before
    if (C > 1) {
        int g = 0, e = 0;
        for (int q0 = 0; q0 < m; q0 += kBatch) {
            uint32_t key[kFly];
            batch(q0, key);
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                if (live(q0, u)) {
                    g += above_it(key[u]) ? 1 : 0;
                    e += equal_it(key[u]) ? 1 : 0;
                }
        }
        g = __reduce_add_sync(0xffffffffu, g);
        e = __reduce_add_sync(0xffffffffu, e);
        if (lane == 0) {
            atomicAdd(&mine.x, g);
            atomicAdd(&mine.y, e);
        }
        __syncthreads();
        if (tid < C)
            cluster.map_shared_rank(before, tid)[rank] = mine;
        cluster.sync();                              // the last access to another block's memory
        for (int r = 0; r < rank; ++r) {
            above += before[r].x;
            equal += before[r].y;
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int q0 = 0; q0 < m; q0 += kBatch) {
        uint32_t key[kFly], g[kFly], e[kFly];
        batch(q0, key);
        __syncthreads();                             // the batch before has read tally
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            g[u] = __ballot_sync(0xffffffffu, live(q0, u) && above_it(key[u]));
            e[u] = __ballot_sync(0xffffffffu, live(q0, u) && equal_it(key[u]));
            if (lane == 0)
                tally[u * kSelWarps + warp] = __popc(g[u]) | (__popc(e[u]) << 16);
        }
        __syncthreads();
        // Every warp sums all tallies, four a lane (4096 keys: each half fits).
        const int4 t = reinterpret_cast<const int4*>(tally)[lane];
        const int sum = t.x + t.y + t.z + t.w;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        const int excl = incl - sum;
        const int entry = warp & 3;                  // of the four of lane u * 4 + warp / 4
        const int mid = excl + (entry > 0 ? t.x : 0) + (entry > 1 ? t.y : 0) + (entry > 2 ? t.z : 0);
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const int at = __shfl_sync(0xffffffffu, mid, u * (kSelWarps / 4) + (warp >> 2));
            const int ga = above + (at & 0xffff) + __popc(g[u] & below);
            const int ea = equal + (at >> 16) + __popc(e[u] & below);
            const bool eq = e[u] >> lane & 1u;
            if ((g[u] >> lane & 1u) || (eq && ea < want))
                kept[a.sinks + ga + (ea < want ? ea : want)] = lo + q0 + u * kSelThreads + tid;
        }
        const int sums = __shfl_sync(0xffffffffu, incl, 31);
        above += sums & 0xffff;
        equal += sums >> 16;
    }
}

constexpr int kMoveThreads = 256;
constexpr int kInPlaceSlice = 64;            // bytes of a row per block, in place
constexpr int kUnroll = 4;                   // rows of a tile per thread
constexpr int kTableInts = 6 * 1024;         // page ids staged in shared memory
constexpr int kChunkBytes = 256 * 1024;      // of K or V per block, where the order is free
// Rows of one tile, for slices of `slice` bytes.
__host__ __device__ constexpr int tile_rows(int slice) { return kMoveThreads / (slice / 16) * kUnroll; }

// How a move kernel's blocks take the rows of their (request, KV head): all of
// them in order (in place), a chunk of them, or one tile of them.
enum MoveKind : int { kInPlace, kChunk, kTile };

// Rows [j_begin, j_end) of the kept ones. T: uint4 with kPerRow threads per row
// slice, or float with one (the weights). bt, dt: the request's page ids. One
// tile is in registers while the next one's rows are read, and the positions of
// the one after are on their way. A row's source is never a destination of an
// earlier tile, so reading ahead is safe; in place, the barrier keeps a tile's
// writes behind every thread's reads of it.
template <typename T, int kPerRow, MoveKind kKind>
__device__ __forceinline__ void move_rows(const EvictArgs& a, T* pool, int64_t row_units, int unit,
                                          const int32_t* bt, const int32_t* dt, int h, int j_begin,
                                          int j_end, const int32_t* kept)
{
    constexpr int kRows = kMoveThreads / kPerRow;
    constexpr int kStep = kRows * kUnroll;
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
    if constexpr (kKind == kTile) {          // no more rows than a step of either type
        write(j_begin, 0);
        return;
    }
    fetch(j_begin + kStep);
    for (int j0 = j_begin; j0 < j_end; j0 += 2 * kStep) {
        read(j0 + kStep, 1);
        fetch(j0 + 2 * kStep);
        if (kKind == kInPlace)
            __syncthreads();
        write(j0, 0);
        read(j0 + 2 * kStep, 0);
        fetch(j0 + 3 * kStep);
        if (kKind == kInPlace)
            __syncthreads();
        write(j0 + kStep, 1);
    }
}

// Blocks of a (request, KV head): a column slice of K or of V, or the weights. In
// place the slices are narrow, since a block takes all rows and only the slices
// spread the work (8192 rows of 64 heads: 131 us with 64 bytes, 159 with 128, 152 with
// 32; e4m3 rows of 128 bytes 108, 150 and 91); where the order is free they are whole
// rows (113 us, 124 with 64 bytes).
template <MoveKind kKind, int kSlice>
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictArgs a)
{
    __shared__ int32_t table[kKind == kTile ? 2 : kTableInts];
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = 2 * a.slices + 1;                // K slices, V slices, the weights
    int64_t blk = blockIdx.x;
    const int part = int(blk % per);
    blk /= per;
    const int chunk = kKind == kInPlace ? 0 : int(blk % a.chunks);
    const int64_t bh = kKind == kInPlace ? blk : blk / a.chunks;
    const int b = int(bh / a.H_kv), h = int(bh - int64_t(b) * a.H_kv);
    const int n = evict_context(a, b, false);
    const int len = n < a.keep ? n : a.keep;
    const int32_t* kept = a.kept + bh * a.keep;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int32_t* dt = a.dst_table + int64_t(b) * a.dst_max_pages;
    const int j_begin = chunk * a.chunk_rows;
    const int j_end = kKind == kInPlace ? len : min(len, j_begin + a.chunk_rows);
    if (j_begin >= j_end)
        return;
    const int d0 = j_begin >> a.ps_shift, d1 = (j_end - 1) >> a.ps_shift;
    if constexpr (kKind != kInPlace) {
        // A destination that the request still reads: recorded, and the block's
        // rows are not written.
        int own = 0;
        for (int i = d0 + int(threadIdx.x); i <= d1; i += kMoveThreads)
            own |= dt[i] == bt[i];
        if (__syncthreads_or(own)) {
            if (threadIdx.x == 0)
                atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
            return;
        }
    }
    if constexpr (kKind != kTile) {
        // The page ids of these rows in shared memory, where they fit.
        const int s0 = kept[j_begin] >> a.ps_shift, s1 = kept[j_end - 1] >> a.ps_shift;
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
    }
    if (part == 2 * a.slices) {
        move_rows<float, 1, kKind>(a, a.weight_pages, 1, 0, bt, dt, h, j_begin, j_end, kept);
    } else {
        const bool is_v = part >= a.slices;
        const int slice = part - (is_v ? a.slices : 0);
        move_rows<uint4, kSlice / 16, kKind>(
            a, static_cast<uint4*>(is_v ? a.value_pages : a.key_pages), a.row_bytes / 16,
            slice * (kSlice / 16) + int(threadIdx.x % (kSlice / 16)), bt, dt, h, j_begin, j_end, kept);
    }
}

}  // namespace

cudaError_t launch_evict(EvictArgs a, int device, int sm_count, cudaStream_t stream)
{
    const int64_t heads = int64_t(a.B) * a.H_kv;
    const int64_t cap = int64_t(a.max_pages) << a.ps_shift;
    const int64_t rows = cap < a.keep ? cap : a.keep;
    const bool in_place = a.dst_table == a.block_table;
    const int slice = in_place ? kInPlaceSlice : a.row_bytes;
    a.slices = a.row_bytes / slice;
    const int64_t parts = heads * (2 * a.slices + 1);
    // Chunks of kChunkBytes, of less (down to a tile) while that leaves the GPU
    // short of blocks.
    a.chunk_rows = kChunkBytes / slice;
    while (a.chunk_rows > tile_rows(slice) &&
           parts * ((rows + a.chunk_rows - 1) / a.chunk_rows) < 3 * int64_t(sm_count))
        a.chunk_rows /= 2;
    a.chunks = in_place ? 1 : int((rows + a.chunk_rows - 1) / a.chunk_rows);
    const int64_t moves = parts * a.chunks;
    // Blocks per (request, KV head) for the choice: more while the GPU has room
    // for them (two per SM) and each still has more than a batch of keys.
    int C = 1;
    while (C < kMaxCluster && heads * C * 2 <= 2 * int64_t(sm_count) && cap > int64_t(kBatch) * C)
        C *= 2;
    if (moves >= (int64_t(1) << 31) || heads * C >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    // whole batches of keys in shared memory
    const int64_t share = ((cap + C - 1) / C + 31 + kBatch - 1) / kBatch * kBatch;
    const int cached = int(share < kSelKeys ? share : kSelKeys);
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev];
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    cudaError_t e;
    if (!raised[device].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (2 * kBins + kSelKeys) * int(sizeof(uint32_t)));
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
    cfg.dynamicSmemBytes = size_t(2 * kBins + cached) * sizeof(uint32_t);
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
    const bool tile = a.chunk_rows == tile_rows(slice), wide = slice == 256;
    return cudaLaunchKernelEx(&cfg,
                              in_place ? evict_move_kernel<kInPlace, kInPlaceSlice>
                              : tile   ? (wide ? evict_move_kernel<kTile, 256> : evict_move_kernel<kTile, 128>)
                                       : (wide ? evict_move_kernel<kChunk, 256> : evict_move_kernel<kChunk, 128>),
                              a);
}

}  // namespace pa
