// Split-KV paged attention for few query rows (G * L <= 16 rows per request and
// KV head), for the calls with a sliding window and those that keep their
// scores.
//
// Per row r of a (request, KV head) and its visible keys j:
//   s_rj = c q_r . k_j,  m = max s,  l = sum 2^(s - m),  o = sum 2^(s - m) v_j / l
// in the log2 domain (c = scale log2 e), by the online recurrence.
//
// The keys, not the query rows, are the tall side of both matrix products:
// S^T = K Q^T (16 keys x 8 rows per mma) and O^T += V^T P^T (16 of D x 8 rows), so
// that a group of up to 8 rows fills the instruction's narrow side. (With the
// rows on the tall side, as in the many-row kernel, 4 rows fill a quarter of
// it and the e4m3 form was bound by its instructions.)
//
//   * Both sums run over an index whose order is free, so 16 contiguous bytes of
//     a row are the very words that a lane's instructions want: K with four
//     lanes a row, V with eight, V's pairs of keys joined by byte permutes.
//   * Each warp has a ring of its own, two tiles (16 KiB) deep, that it fills by
//     TMA (whole page slices, 128-byte swizzle) and empties itself: 128 KiB on
//     their way per SM, across the ends of pieces, and no barrier between the
//     warps but at the end of a piece. (Copies by the lanes themselves, into
//     registers or shared memory, came to 4.1-4.6 TB/s however many were
//     issued.)
//   * P is split into two bf16 parts (their sum has 16 bits), so its rounding
//     does not show next to the output's; the tensor core has the time. e4m3
//     pages: codes become f16 exactly, P is one f16.
//   * The maximum in use moves only when a score exceeds it by 2^8 (P stays
//     below 2^8, the softmax is the same), so the common step needs one vote
//     instead of a shuffle tree.
//   * The tiles of all (request, KV head) form one stream of granules (one tile
//     for each of a block's four warps) that the grid splits evenly, as the
//     many-row kernel does; a piece that does not hold its whole segment leaves
//     its state in the workspace, and a second, small kernel merges the pieces
//     in their order.
//
// Bound by memory: every K and V byte that a row sees is read once. Measured (one
// call of a replayed graph): 64 bf16 requests, window 2048, 508 MB in 85 us
// (6.0 TB/s, of 6.8 measured for a copy); e4m3, 255 MB in 49 us; 32 requests of
// a window of 1024 in groups of 7, 51 MB in 16 us; one request, window 512, 8.2
// us, of which the second kernel is about 3.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_split.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kMoveLog2 = 8.f;      // scores may exceed the maximum in use by this much
constexpr int kPieceUnits = 1;        // a piece's cost beyond its granules
// Two blocks of two tiles a warp. 64 e4m3 requests, window 2048: 49 us, with three
// blocks 62, with four tiles a warp 75; 8 bf16 requests of 16k-32k: 142, 160 and
// 189. (Presumably the second kernel's blocks and the next call's then find no
// room until the last block of this one ends.)
constexpr int kBlocksPerSM = 2;

// kTok keys per step and warp: 16 rows of 256 bytes or 32 of 128.
template <int D, bool F8>
struct Shape {
    static constexpr int kRowBytes = D * (F8 ? 1 : 2);
    static constexpr int kTok = kRowBytes == 256 ? 16 : 32;
    static constexpr int kSub = kTok / 16;
    static constexpr int kKLoads = kRowBytes / 64;    // 16-byte loads per lane and K row
    static constexpr int kVLoads = kRowBytes / 128;   // and V row
    static constexpr int kSteps = D / 16;             // k-steps of S, 16-row tiles of O^T
};

constexpr int kStages = 2;            // tiles on their way per warp
constexpr int kTileBytes = 4096;      // K (or V) of one tile: [128-byte column block][key][128 bytes]
template <int D, int NT>
struct Smem {
    static constexpr int kSlab = (D / 16 * NT * 4 + 4 * NT) * 32 * 4; // one warp's state: O^T, m, l
    static constexpr int kRing = 0;                                   // [warp][stage][K, V]
    static constexpr int kSlabs = kRing + kWarps * kStages * 2 * kTileBytes;
    static constexpr int kBars = kSlabs + 2 * kSlab;                  // [warp][stage][K, V]
    static constexpr int kMisc = kBars + kWarps * kStages * 2 * 8;
    static constexpr int kPrefix = kMisc + 16;                        // [B + 1] granules before, [B] granules, [B] lengths
    static size_t bytes(int B) { return kPrefix + size_t(3 * B + 1) * 4 + 1024; }
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The tiles of kTok keys that a request of n tokens visits: with a window those
// of [0, sinks), then those from `start`, the first key that some row sees
// through the window (first_seen) rounded down to a page (or a tile within a
// larger one); one run from 0 where the two would meet.
struct TileSpan {
    int sink_tiles, start, first_seen, granules;
};
template <int kTok, int kMode>
__device__ __forceinline__ TileSpan tile_span(const DecodeArgs& a, int n)
{
    TileSpan s{0, 0, 0, 0};
    if constexpr (kMode == kWindow) {
        s.first_seen = int(max(int64_t(0), int64_t(n) - a.L - a.window + 1));
        const int start = s.first_seen & ~(a.box_rows - 1);
        if (start > a.sinks) {
            s.sink_tiles = (a.sinks + kTok - 1) / kTok;
            s.start = start;
        }
    }
    const int tiles = s.sink_tiles + (n - s.start + kTok - 1) / kTok;
    s.granules = max(1, (tiles + kWarps - 1) / kWarps);
    return s;
}

template <int kMode>
__device__ __forceinline__ int context_cap(const DecodeArgs& a)
{
    const int cap = a.max_pages * a.ps;
    return kMode == kScores ? min(cap, a.score_cap) : cap;
}

// The softmax state of up to 8 NT rows in one warp's lanes: O^T as the tensor
// core leaves it (rows 8 nt + 2 q + (k & 1)), and m and l of the lane's rows.
template <int D, int NT>
struct RowState {
    static constexpr int kKS = D / 16;
    static constexpr int kRegs = kKS * NT * 4;
    static constexpr int kPlaces = kRegs + 4 * NT;
    float o[kKS][NT][4], m[NT][2], l[NT][2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < kKS; ++t)
                o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.f;
        }
    }
    // To and from kPlaces x 32 floats, lane by lane.
    __device__ __forceinline__ void put(float* to, int lane) const
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int t = 0; t < kKS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    to[((nt * kKS + t) * 4 + k) * 32 + lane] = o[t][nt][k];
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                to[(kRegs + 4 * nt + rr) * 32 + lane] = m[nt][rr];
                to[(kRegs + 4 * nt + 2 + rr) * 32 + lane] = l[nt][rr];
            }
        }
    }
    // M = max, l = l 2^(m - M) + l' 2^(m' - M), likewise O.
    __device__ __forceinline__ void fold(const float* v)
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f1[2], f2[2];
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const float m2 = v[kRegs + 4 * nt + rr], l2 = v[kRegs + 4 * nt + 2 + rr];
                const float M = fmaxf(m[nt][rr], m2);
                f1[rr] = m[nt][rr] == -INFINITY ? 0.f : fast_exp2(m[nt][rr] - M);
                f2[rr] = m2 == -INFINITY ? 0.f : fast_exp2(m2 - M);
                m[nt][rr] = M;
                l[nt][rr] = l[nt][rr] * f1[rr] + l2 * f2[rr];
            }
#pragma unroll
            for (int t = 0; t < kKS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[t][nt][k] = o[t][nt][k] * f1[k & 1] + v[(nt * kKS + t) * 4 + k] * f2[k & 1];
        }
    }
    __device__ __forceinline__ void take(const float* from, int lane)
    {
        float v[kPlaces];
#pragma unroll
        for (int i = 0; i < kPlaces; ++i)
            v[i] = from[i * 32 + lane];
        fold(v);
    }
    // Four warps' states into warp 0's: 2 and 3 into 0 and 1, then 1 into 0.
    // slabs: two states; free when the block comes here. By the whole block.
    __device__ __forceinline__ void gather(float* slabs, int warp, int lane)
    {
        if (warp >= 2)
            put(slabs + (warp - 2) * kPlaces * 32, lane);
        __syncthreads();
        if (warp < 2)
            take(slabs + warp * kPlaces * 32, lane);
        if (warp == 1)
            put(slabs + kPlaces * 32, lane);
        __syncthreads();
        if (warp == 0)
            take(slabs + kPlaces * 32, lane);
    }
    // The output rows of (request, KV head) bh, from q_row0 on: each lane holds
    // runs of neighbouring elements of D.
    template <bool F8, int kMode>
    __device__ __forceinline__ void write(const DecodeArgs& a, int64_t bh, int64_t q_row0, int lane) const
    {
        const int g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = 8 * nt + 2 * q + rr;
                if (r >= a.R)
                    continue;
                if constexpr (kMode == kScores) {
                    if (g == 0)
                        a.row_state[bh * a.R + r] = make_float2(m[nt][rr], l[nt][rr]);
                }
                const float inv = l[nt][rr] > 0.f ? a.v_scale / l[nt][rr] : 0.f;
                uint16_t* dst = a.out + (q_row0 + r) * D;
                auto pair = [&](int t, int k) { return pack_bf16x2(o[t][nt][k] * inv, o[t + 1][nt][k] * inv); };
                if constexpr (D == 64) {             // element 8 g + t + 4 half
                    *reinterpret_cast<uint4*>(dst + 8 * g) =
                        make_uint4(pair(0, rr), pair(2, rr), pair(0, 2 + rr), pair(2, 2 + rr));
                } else {                             // e4m3: 16 g + t + 8 half; bf16: 64 half + 8 g + t
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = 2 * half + rr;
                        *reinterpret_cast<uint4*>(dst + (F8 ? 16 * g + 8 * half : 64 * half + 8 * g)) =
                            make_uint4(pair(0, k), pair(2, k), pair(4, k), pair(6, k));
                    }
                }
            }
    }
};

template <int D, bool F8, int NT, int kMode>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM)
    decode_rows_kernel(const __grid_constant__ CUtensorMap key_map,
                       const __grid_constant__ CUtensorMap value_map, const DecodeArgs a)
{
    using Sh = Shape<D, F8>;
    using Lay = Smem<D, NT>;
    constexpr int kTok = Sh::kTok, kSub = Sh::kSub, kKL = Sh::kKLoads, kVL = Sh::kVLoads, kKS = Sh::kSteps;
    constexpr int kSlot = Lay::kSlab / 4;             // floats of a piece's state
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int* misc = reinterpret_cast<volatile int*>(smem + Lay::kMisc);
    int32_t* pre = reinterpret_cast<int32_t*>(smem + Lay::kPrefix);
    int32_t* gbr = pre + a.B + 1;
    int32_t* len = gbr + a.B;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int per_req = a.H_kv;
    const int cap = context_cap<kMode>(a);
    const float c = a.scale_log2;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBars) + warp * kStages * 2;
    if (lane == 0) {
        for (int i = 0; i < kStages * 2; ++i)
            mbar_init(&bars[i], 1);
        if (warp == 0) {
            misc[0] = 0;                              // a wait ran out
            prefetch_tensormap(&key_map);
            prefetch_tensormap(&value_map);
        }
        fence_barrier_init();
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this block's granules [x_begin, x_end) -------------------------------
    if (warp == 0) {
        int carry = 0;
        if (lane == 0)
            pre[0] = 0;
        for (int base = 0; base < a.B; base += 32) {
            const int b = base + lane;
            int gs = 0;
            if (b < a.B) {
                const int n = clamp_context(a.context_lens[b], cap, a.err);
                gs = tile_span<kTok, kMode>(a, n).granules;
                gbr[b] = gs;
                len[b] = n;
            }
            int incl = gs * per_req;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            if (b < a.B)
                pre[b + 1] = carry + incl;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
    const int64_t units = pre[a.B] + int64_t(kPieceUnits) * a.B * per_req;
    const int64_t grid = int64_t(gridDim.x) < units ? int64_t(gridDim.x) : units;
    const int64_t cta = blockIdx.x;
    if (cta >= grid)
        return;
    StreamPoint p0, p1;
    granules_at_units(pre, gbr, a.B, per_req, udiv64(cta * units, grid), udiv64((cta + 1) * units, grid),
                      units, kPieceUnits, p0, p1);
    if (p0.x >= p1.x)
        return;
    const int64_t x_end = p1.x;

    // A place in the stream, with what its segment needs: the loads run ahead of
    // the products, across the ends of pieces.
    struct Place {
        int64_t x;
        SegmentPos sp;
        int n;
        TileSpan span;
    };
    auto enter = [&](Place& p) {
        p.n = len[p.sp.b];
        p.span = tile_span<kTok, kMode>(a, p.n);
    };
    // First token of the warp's tile of place p, and the end of its run.
    auto tile_at = [&](const Place& p, int* end) {
        const int t = int(p.x - p.sp.seg_start) * kWarps + warp;
        const bool first_run = kMode == kWindow && t < p.span.sink_tiles;
        *end = first_run ? a.sinks : p.n;
        return first_run ? t * kTok : p.span.start + (t - p.span.sink_tiles) * kTok;
    };
    // A tile is copied in boxes of box_rows keys of one page, box j by lane j:
    // whether a row sees a key of it, the page id (requested a step before its
    // use), and the box's row in the pool.
    const int box_shift = __ffs(a.box_rows) - 1;
    auto box_token = [&](const Place& p) {
        int end;
        const int t = tile_at(p, &end) + (lane << box_shift);
        const bool live = (lane << box_shift) < kTok && t < end &&
                          !(kMode == kWindow && t >= a.sinks && t + a.box_rows <= p.span.first_seen);
        return live ? t : -1;
    };
    auto page_of = [&](const Place& p) {
        const int t = box_token(p);
        return t < 0 ? 0 : __ldg(a.block_table + int64_t(p.sp.b) * a.max_pages + (t >> a.ps_shift));
    };
    auto row_of = [&](const Place& p, int phys) {
        const int t = box_token(p);
        if (t < 0)
            return -1;
        if (unsigned(phys) >= unsigned(a.num_pages)) {
            atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
            phys = 0;
        }
        return ((phys * a.H_kv + p.sp.h) << a.ps_shift) + (t & ((1 << a.ps_shift) - 1));
    };
    uint8_t* ring = smem + Lay::kRing + warp * (kStages * 2 * kTileBytes);
    constexpr int kHalves = Sh::kRowBytes / 128;     // 128-byte column blocks of a row
    constexpr int kHalfBytes = kTok * 128;
    const uint64_t policy = l2_policy_evict_first();
    // K (v = 0) or V of the tile whose boxes are at pool rows `row` (-1: none).
    auto copy = [&](int row, int stage, int v) {
        uint64_t* bar = &bars[stage * 2 + v];
        const unsigned who = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0)
            mbar_arrive_expect_tx(bar, uint32_t(__popc(who)) * a.box_rows * Sh::kRowBytes);
        __syncwarp();
        if (row >= 0) {
            uint8_t* dst = ring + (stage * 2 + v) * kTileBytes + (lane << box_shift) * 128;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
                tma_load_2d(dst + hf * kHalfBytes, v ? &value_map : &key_map, hf * 64, row, bar, policy);
        }
    };
    // The next tile to be requested, and its rows (found a step ahead).
    Place ahead;
    ahead.x = p0.x;
    ahead.sp = segment_at(pre, gbr, per_req, 1, p0.b, p0.hm);
    enter(ahead);
    Place at = ahead;                     // the tile at hand
    auto step = [&](Place& p) {
        if (++p.x < x_end && p.x == p.sp.seg_start + p.sp.seg_len) {
            p.sp = next_segment(pre, gbr, per_req, 1, p.sp);
            enter(p);
        }
    };
    int page = page_of(ahead);
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
        const bool live = ahead.x < x_end;
        if (live) {
            const int row = row_of(ahead, page);
            step(ahead);
            if (ahead.x < x_end)
                page = page_of(ahead);
            copy(row, st, 0);
            copy(row, st, 1);
        }
    }
    const int swz = a.swz;                           // 7: swizzled; 0: boxes of fewer than 8 rows
    int stage = 0;
    uint32_t phase = 0;

    while (at.x < x_end) {
        const SegmentPos sp = at.sp;
        const int n = at.n;
        const TileSpan span = at.span;
        const int64_t piece_end = min(x_end, sp.seg_start + sp.seg_len);
        const int64_t q_row0 = (int64_t(sp.b) * a.H_q + sp.h * a.G) * a.L;

        // Query fragments: column n = 8 nt + g of Q^T, the elements of D that
        // this lane's K words hold.
        uint32_t qb[NT][kKS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + (q_row0 + r) * D);
            if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (r < a.R) {
                        w[0] = *reinterpret_cast<const uint4*>(src + 128 * j + 32 * q);
                        w[1] = *reinterpret_cast<const uint4*>(src + 128 * j + 32 * q + 16);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        qb[nt][4 * j + i][0] = bf16x2_to_f16x2(word(w[i >> 1], 2 * (i & 1)));
                        qb[nt][4 * j + i][1] = bf16x2_to_f16x2(word(w[i >> 1], 2 * (i & 1) + 1));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < kKL; ++j) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (r < a.R)
                        w = *reinterpret_cast<const uint4*>(src + 64 * j + 16 * q);
                    qb[nt][2 * j][0] = w.x;
                    qb[nt][2 * j][1] = w.y;
                    qb[nt][2 * j + 1][0] = w.z;
                    qb[nt][2 * j + 1][1] = w.w;
                }
            }
        }
        // Last visible position of this lane's rows 8 nt + 2 q + rr, and the
        // window's first.
        int lim[NT][2], low[NT][2];
        int lim_min = 0x7fffffff, low_max = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = 8 * nt + 2 * q + rr;
                const int i = r < a.R ? r % a.L : a.L - 1;
                lim[nt][rr] = a.causal ? min(n - a.L + i, n - 1) : n - 1;
                low[nt][rr] = lim[nt][rr] - a.window + 1;
                lim_min = min(lim_min, lim[nt][rr]);
                low_max = max(low_max, low[nt][rr]);
            }
        lim_min = __reduce_min_sync(0xffffffffu, lim_min);
        if constexpr (kMode == kWindow)
            low_max = __reduce_max_sync(0xffffffffu, low_max);

        RowState<D, NT> st;
        st.clear();
        auto& m = st.m;
        auto& l = st.l;
        auto& o = st.o;

        for (; at.x < piece_end; ++at.x) {
            int end;
            const int t0 = tile_at(at, &end);
            const bool busy = t0 < end;              // the last granule may hold fewer than four tiles
            const bool first_run =
                kMode == kWindow && int(at.x - sp.seg_start) * kWarps + warp < span.sink_tiles;
            const uint8_t* kt = ring + stage * (2 * kTileBytes);
            const uint8_t* vt = kt + kTileBytes;
            mbar_wait_warp(&bars[stage * 2], phase, misc, a.err);
            // ---- S^T = K Q^T: tokens 16 s + g (+ 8), rows 2 q + {0, 1}
            // (even and odd k-steps apart: half the chain of dependent products)
            float sc[kSub][NT][4], odd[kSub][NT][4];
#pragma unroll
            for (int s = 0; s < kSub; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sc[s][nt][k] = odd[s][nt][k] = 0.f;
            if (busy) {
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    uint4 kr[2][kKL];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int i = 0; i < kKL; ++i)
                            kr[hh][i] = *reinterpret_cast<const uint4*>(
                                kt + (i >> 1) * kHalfBytes + (16 * s + 8 * hh + g) * 128 +
                                (((4 * (i & 1) + q) ^ (g & swz)) << 4));
#pragma unroll
                    for (int ks = 0; ks < kKS; ++ks) {
                        uint32_t A[4];
                        if constexpr (F8) {
                            const uint32_t w0 = word(kr[0][ks >> 2], ks & 3), w1 = word(kr[1][ks >> 2], ks & 3);
                            A[0] = e4m3x2_to_f16x2(w0);
                            A[1] = e4m3x2_to_f16x2(w1);
                            A[2] = e4m3x2_hi_to_f16x2(w0);
                            A[3] = e4m3x2_hi_to_f16x2(w1);
                        } else {
                            A[0] = word(kr[0][ks >> 1], 2 * (ks & 1));
                            A[1] = word(kr[1][ks >> 1], 2 * (ks & 1));
                            A[2] = word(kr[0][ks >> 1], 2 * (ks & 1) + 1);
                            A[3] = word(kr[1][ks >> 1], 2 * (ks & 1) + 1);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float* d = ks & 1 ? odd[s][nt] : sc[s][nt];
                            if constexpr (F8)
                                mma_f16_16816(d, A, qb[nt][ks][0], qb[nt][ks][1]);
                            else
                                mma_bf16_16816(d, A, qb[nt][ks][0], qb[nt][ks][1]);
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < kSub; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sc[s][nt][k] += odd[s][nt][k];
            }
            // The keys of the tile kStages on (into the place just read), and the
            // rows of the one after.
            int row_v = -1;
            const bool more = ahead.x < x_end;
            if (more) {
                row_v = row_of(ahead, page);
                __syncwarp();                        // every lane has read the place
                copy(row_v, stage, 0);
                step(ahead);
                if (ahead.x < x_end)
                    page = page_of(ahead);
            }
            const bool edge = t0 + kTok - 1 > lim_min || t0 + kTok > end || (kMode == kWindow && t0 < low_max);
            if (busy) {
                if (edge) {
#pragma unroll
                    for (int s = 0; s < kSub; ++s)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int tok = t0 + 16 * s + g + 8 * (j >> 1);
                                bool seen = tok < end && tok <= lim[nt][j & 1];
                                if constexpr (kMode == kWindow)
                                    seen = seen && (tok < a.sinks || (!first_run && tok >= low[nt][j & 1]));
                                if (!seen)
                                    sc[s][nt][j] = -INFINITY;
                            }
                }
                if constexpr (kMode == kScores) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const int r = 8 * nt + 2 * q + rr;
                            if (r < a.R) {
                                float* to = a.scores + ((int64_t(sp.b) * a.H_kv + sp.h) * a.R + r) * a.score_stride +
                                            t0 + g;
#pragma unroll
                                for (int s = 0; s < kSub; ++s) {
                                    to[16 * s] = sc[s][nt][rr] * c;
                                    to[16 * s + 8] = sc[s][nt][2 + rr] * c;
                                }
                            }
                        }
                }
                // ---- the maximum in use
                float mx[NT][2];
                bool moves = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                        float v = fmaxf(sc[0][nt][rr], sc[0][nt][2 + rr]);
#pragma unroll
                        for (int s = 1; s < kSub; ++s)
                            v = fmaxf(v, fmaxf(sc[s][nt][rr], sc[s][nt][2 + rr]));
                        mx[nt][rr] = v * c;
                        moves |= mx[nt][rr] > m[nt][rr] + kMoveLog2 ||
                                 (m[nt][rr] == -INFINITY && mx[nt][rr] > -INFINITY);
                    }
                if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            float v = mx[nt][rr];
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1)
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                            if (v > m[nt][rr]) {
                                const float f = m[nt][rr] == -INFINITY ? 0.f : fast_exp2(m[nt][rr] - v);
                                m[nt][rr] = v;
                                l[nt][rr] *= f;
#pragma unroll
                                for (int t = 0; t < kKS; ++t) {
                                    o[t][nt][rr] *= f;
                                    o[t][nt][2 + rr] *= f;
                                }
                            }
                        }
                }
                // ---- P^T: two keys of one row a register, after the transpose
                uint32_t ph[kSub][NT][2], pl[kSub][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float mu[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0],
                                         m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
#pragma unroll
                    for (int s = 0; s < kSub; ++s)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const float p0v = fast_exp2(fmaf(sc[s][nt][2 * hh], c, -mu[0]));
                            const float p1v = fast_exp2(fmaf(sc[s][nt][2 * hh + 1], c, -mu[1]));
                            l[nt][0] += p0v;
                            l[nt][1] += p1v;
                            if constexpr (F8) {
                                ph[s][nt][hh] = transpose8x8(pack_f16x2(p0v, p1v));
                            } else {
                                const uint32_t hi = pack_bf16x2(p0v, p1v);
                                ph[s][nt][hh] = transpose8x8(hi);
                                pl[s][nt][hh] = transpose8x8(pack_bf16x2(p0v - __uint_as_float(hi << 16),
                                                                         p1v - __uint_as_float(hi & 0xffff0000u)));
                            }
                        }
                }
                // ---- O^T += V^T P^T; tile t of O^T holds the elements of D that the
                // lanes' words give to it (RowState::write has them in order)
                mbar_wait_warp(&bars[stage * 2 + 1], phase, misc, a.err);
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    uint4 vr[4][kVL];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 16 * s + 2 * q + (k & 1) + 8 * (k >> 1);
#pragma unroll
                        for (int i = 0; i < kVL; ++i)
                            vr[k][i] = *reinterpret_cast<const uint4*>(vt + i * kHalfBytes + r * 128 +
                                                                       ((g ^ (r & swz)) << 4));
                    }
                    if (edge) {
                        // Keys that no row sees: zeros, whatever the page holds (P is 0
                        // there, but 0 * NaN is not).
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tok = t0 + 16 * s + 2 * q + (k & 1) + 8 * (k >> 1);
                            if (tok >= end || (kMode == kWindow && tok >= a.sinks && tok < span.first_seen))
#pragma unroll
                                for (int i = 0; i < kVL; ++i)
                                    vr[k][i] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    auto product = [&](int t, const uint32_t* A) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (F8) {
                                mma_f16_16816(o[t][nt], A, ph[s][nt][0], ph[s][nt][1]);
                            } else {
                                mma_bf16_16816(o[t][nt], A, ph[s][nt][0], ph[s][nt][1]);
                                mma_bf16_16816(o[t][nt], A, pl[s][nt][0], pl[s][nt][1]);
                            }
                        }
                    };
                    if constexpr (F8) {
                        // word w: codes 4 w .. 4 w + 3 (rows g of tiles), w + 2: rows g + 8
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            uint32_t f[2][2][4];      // [keys 2 q / 2 q + 8][half][element of the word]
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                                for (int hh = 0; hh < 2; ++hh) {
                                    const uint32_t x0 = word(vr[2 * kk][0], w + 2 * hh);
                                    const uint32_t x1 = word(vr[2 * kk + 1][0], w + 2 * hh);
                                    const uint32_t e01 = __byte_perm(x0, x1, 0x5140);
                                    const uint32_t e23 = __byte_perm(x0, x1, 0x7362);
                                    f[kk][hh][0] = e4m3x2_to_f16x2(e01);
                                    f[kk][hh][1] = e4m3x2_hi_to_f16x2(e01);
                                    f[kk][hh][2] = e4m3x2_to_f16x2(e23);
                                    f[kk][hh][3] = e4m3x2_hi_to_f16x2(e23);
                                }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t A[4] = {f[0][0][e], f[0][1][e], f[1][0][e], f[1][1][e]};
                                product(4 * w + e, A);
                            }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < kKS; ++t) {
                            // elements e0 (rows g) and e1 (rows g + 8) of a lane's words
                            constexpr bool kTwo = D == 128;
                            const int e0 = t, e1 = kTwo ? t : t + 4;
                            uint32_t A[4];
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk) {
                                A[2 * kk] = __byte_perm(word(vr[2 * kk][0], e0 >> 1), word(vr[2 * kk + 1][0], e0 >> 1),
                                                        e0 & 1 ? 0x7632 : 0x5410);
                                A[2 * kk + 1] =
                                    __byte_perm(word(vr[2 * kk][kTwo ? 1 : 0], e1 >> 1),
                                                word(vr[2 * kk + 1][kTwo ? 1 : 0], e1 >> 1), e1 & 1 ? 0x7632 : 0x5410);
                            }
                            product(t, A);
                        }
                    }
                }
            } else {
                mbar_wait_warp(&bars[stage * 2 + 1], phase, misc, a.err);   // nothing was copied
            }
            if (more) {
                __syncwarp();
                copy(row_v, stage, 1);
            }
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }

        // ---- end of a piece ---------------------------------------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][rr] += __shfl_xor_sync(0xffffffffu, l[nt][rr], off);
        __syncthreads();                             // the piece before has read the slabs
        st.gather(reinterpret_cast<float*>(smem + Lay::kSlabs), warp, lane);
        if (warp == 0 && !misc[0]) {
            if (sp.seg_start >= p0.x && sp.seg_start + sp.seg_len <= x_end)
                st.template write<F8, kMode>(a, int64_t(sp.b) * a.H_kv + sp.h, q_row0, lane);
            else                                     // a slot of its own: segment and block
                st.put(a.partials + (int64_t(sp.seg) + cta) * kSlot, lane);
        }
        // on to the next segment
        if (at.x < x_end) {
            at.sp = next_segment(pre, gbr, per_req, 1, sp);
            enter(at);
        }
    }
}

// The segments that straddle blocks: one block each (the others return once the
// first kernel is done). Warp w folds pieces w, w + 4, ... in order, one on its
// way while the one before is folded in.
template <int D, bool F8, int NT, int kMode>
__global__ void __launch_bounds__(kThreads) decode_rows_merge_kernel(const DecodeArgs a, int decode_grid)
{
    using Sh = Shape<D, F8>;
    using State = RowState<D, NT>;
    constexpr int kSlot = State::kPlaces * 32;
    __shared__ float slabs[2 * kSlot];
    __shared__ int red[2][kWarps];
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seg = blockIdx.x;
    const int b = seg / a.H_kv, h = seg - b * a.H_kv;
    const int cap = context_cap<kMode>(a);
    auto granules = [&](int r) {
        const int n = __ldcg(a.context_lens + r);
        return tile_span<Sh::kTok, kMode>(a, n < 0 ? 0 : n > cap ? cap : n).granules;
    };
    // The split of the first kernel, from its inputs (which were complete before
    // it let this one start).
    int before = 0, total = 0;
    for (int r = threadIdx.x; r < a.B; r += kThreads) {
        const int gs = granules(r) * a.H_kv;
        total += gs;
        before += r < b ? gs : 0;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
        red[0][warp] = total;
        red[1][warp] = before;
    }
    __syncthreads();
    total = before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        total += red[0][w];
        before += red[1][w];
    }
    const int len = granules(b);
    const int64_t units = total + int64_t(kPieceUnits) * a.B * a.H_kv;
    const int64_t grid = int64_t(decode_grid) < units ? int64_t(decode_grid) : units;
    const int64_t u0 = before + int64_t(h) * len + int64_t(kPieceUnits) * (seg + 1);
    const int64_t first = block_of_unit(u0, units, grid);
    const int np = int(block_of_unit(u0 + len - 1, units, grid) - first) + 1;
    // Every block waits, so that this grid does not end before the one it
    // follows.
    grid_dependency_wait();
    if (np == 1)
        return;
    const float* slots = a.partials + (int64_t(seg) + first) * kSlot + lane;
    State st;
    st.clear();
    float v[2][State::kPlaces];
    auto fetch = [&](int k, float* to) {
#pragma unroll
        for (int i = 0; i < State::kPlaces; ++i)
            to[i] = __ldcg(slots + int64_t(k) * kSlot + i * 32);
    };
    if (warp < np)
        fetch(warp, v[0]);
    for (int k = warp; k < np; k += 2 * kWarps) {
        if (k + kWarps < np)
            fetch(k + kWarps, v[1]);
        st.fold(v[0]);
        if (k + 2 * kWarps < np)
            fetch(k + 2 * kWarps, v[0]);
        if (k + kWarps < np)
            st.fold(v[1]);
    }
    st.gather(slabs, warp, lane);
    if (warp == 0)
        st.template write<F8, kMode>(a, seg, (int64_t(b) * a.H_q + h * a.G) * a.L, lane);
}

using RowsKernel = void (*)(CUtensorMap, CUtensorMap, DecodeArgs);
using RowsMerge = void (*)(DecodeArgs, int);
struct RowsKernels {
    RowsKernel main;
    RowsMerge merge;
};
template <int D, bool F8, int NT>
RowsKernels rows_kernels(int mode)
{
    if (mode == kWindow)
        return {decode_rows_kernel<D, F8, NT, kWindow>, decode_rows_merge_kernel<D, F8, NT, kWindow>};
    return {decode_rows_kernel<D, F8, NT, kScores>, decode_rows_merge_kernel<D, F8, NT, kScores>};
}
RowsKernels rows_kernels_for(int D, bool fp8, int NT, int mode, int* index)
{
    *index = ((fp8 ? 0 : D == 64 ? 2 : 4) + NT - 1) * 2 + (mode == kWindow ? 0 : 1);
    if (fp8)
        return NT == 1 ? rows_kernels<128, true, 1>(mode) : rows_kernels<128, true, 2>(mode);
    if (D == 64)
        return NT == 1 ? rows_kernels<64, false, 1>(mode) : rows_kernels<64, false, 2>(mode);
    return NT == 1 ? rows_kernels<128, false, 1>(mode) : rows_kernels<128, false, 2>(mode);
}

size_t rows_smem_bytes(int D, int NT, int B)
{
    return D == 64 ? (NT == 1 ? Smem<64, 1>::bytes(B) : Smem<64, 2>::bytes(B))
                   : (NT == 1 ? Smem<128, 1>::bytes(B) : Smem<128, 2>::bytes(B));
}

int row_tiles(const pa_shape& s) { return int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len <= 8 ? 1 : 2; }

}  // namespace

bool decode_rows_takes(const pa_shape& s, int max_smem)
{
    const int64_t R = int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len;
    return R <= 16 && rows_smem_bytes(s.head_dim, row_tiles(s), s.batch) <= size_t(max_smem);
}

int decode_rows_grid(int sm_count) { return sm_count * kBlocksPerSM; }

int decode_rows_box(const pa_shape& s, bool fp8, int page_size)
{
    const int tok = s.head_dim * (fp8 ? 1 : 2) == 256 ? 16 : 32;
    return page_size < tok ? page_size : tok;
}

size_t decode_rows_workspace_bytes(const pa_shape& s, int sm_count)
{
    const int NT = row_tiles(s);
    const size_t slot = s.head_dim == 64 ? (NT == 1 ? Smem<64, 1>::kSlab : Smem<64, 2>::kSlab)
                                         : (NT == 1 ? Smem<128, 1>::kSlab : Smem<128, 2>::kSlab);
    return (size_t(s.batch) * s.num_kv_heads + size_t(decode_rows_grid(sm_count))) * slot;
}

cudaError_t launch_decode_rows(const CUtensorMap& key_map, const CUtensorMap& value_map, DecodeArgs a,
                               const pa_shape& s, int64_t granule_bound, void* workspace,
                               int device, int sm_count, cudaStream_t stream)
{
    const int NT = row_tiles(s);
    int64_t grid = decode_rows_grid(sm_count);
    // Few granules: two of them a block at least, so that a segment's pieces stay
    // few (one request, window 4096: 11.3 us, 14.0 with one; window 512: 8.4 and 8.2).
    if (granule_bound > 0 && granule_bound < 2 * grid)
        grid = (granule_bound + 2 - 1) / 2;
    a.partials = static_cast<float*>(workspace);
    int index = 0;
    const RowsKernels kern = rows_kernels_for(a.D, a.fp8 != 0, NT, a.mode, &index);
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev][12];
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    const int smem = int(rows_smem_bytes(a.D, NT, a.B));
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern.main), &raised[device][index]);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern.main, key_map, value_map, a);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(unsigned(int64_t(a.B) * a.H_kv));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kern.merge, a, int(grid));
}

}  // namespace pa
