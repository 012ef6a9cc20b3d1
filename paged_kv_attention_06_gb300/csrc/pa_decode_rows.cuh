// Split-KV paged attention for few query rows (G * L <= 16 rows per request and
// KV head): the calls with a sliding window, those that keep their scores, the decode
// over 4-bit pools, and a decode's own keys behind a shared prefix (the last two with
// more rows too, in segments of 16).
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
//   * Each warp has a ring of its own, two tiles (16 KiB) deep or one (Smem), that it
//     fills by TMA (whole page slices, 128-byte swizzle; 4-bit rows as they are) and
//     empties itself, across the ends of pieces, and no barrier between the warps but
//     at the end of a piece. On their way per SM: 128 KiB with a window or scores; 96
//     behind a prefix (up to 8 rows; 128 beyond); 60 of 4-bit rows (40). (Copies by the
//     lanes themselves, into registers or shared memory, came to 4.1-4.6 TB/s however
//     many were issued.)
//   * P is split into two bf16 parts (their sum has 16 bits), so its rounding
//     does not show next to the output's; the tensor core has the time. e4m3
//     pages: codes become f16 exactly, P is one f16. 4-bit pages: a value is m + s c;
//     s c becomes an f16 (Q4Step), m goes into the sums by a product of its own with the
//     query's sums over a group (K) and with P (V).
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
// call of a replayed graph): 64 bf16 requests, window 2048, 508 MB in 82 us
// (6.2 TB/s, of 6.7 measured for a copy); e4m3, 255 MB in 47 us; 32 requests of
// a window of 1024 in groups of 7, 51 MB in 16 us; one request, window 512, 8.2
// us, of which the second kernel is about 3.
// 4-bit pools are not: 8 requests of 16k-32k, 244 MB, take 69 us (3.5 TB/s, DRAM at 45 %,
// issue slots at 55 %, tensor pipe at 18 %; e4m3 pools of the same batch 78). A warp's
// tile is one chain of wait, conversion, product, softmax, conversion, product (443
// instructions for 16 keys of K and V), and 12 warps an SM are too few to cover it;
// without any conversion 56 us are left. 32 requests of up to 4096 keys 16, one of 5001 12.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefix.cuh"
#include "pa_q4.cuh"
#include "pa_split.cuh"

namespace pa {
namespace rows {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kMoveLog2 = 8.f;      // scores may exceed the maximum in use by this much
constexpr int kPieceUnits = 1;        // a piece's cost beyond its granules
// Two blocks an SM of two tiles a warp (Smem: not for 4-bit pools, nor behind a prefix). 64
// e4m3 requests, window 2048: 49 us, with three blocks 62, with four tiles a warp 75; 8 bf16
// requests of 16k-32k: 142, 160 and 189. (Presumably the second kernel's blocks and the next
// call's then find no room until the last block of this one ends.)
// kTok keys per step and warp: 16 rows of 256 bytes, 32 of 128, or of 80 (4-bit rows).
template <int D, int KIND>
struct Shape {
    static constexpr int kRowBytes = KIND == kQ4Pool ? kQ4RowBytes : D * (KIND == kE4m3Pool ? 1 : 2);
    static constexpr int kTok = kRowBytes == 256 ? 16 : 32;
    static constexpr int kSub = kTok / 16;
    static constexpr int kKLoads = kRowBytes / 64;    // 16-byte loads per lane and K row
    static constexpr int kVLoads = (kRowBytes + 127) / 128;   // and V row
    static constexpr int kSteps = D / 16;             // k-steps of S, 16-row tiles of O^T
    // K (or V) of one tile: [128-byte column block][key][128 bytes], or [key][80 bytes]
    static constexpr int kTileBytes = kTok * kRowBytes;
};

template <int D, int KIND, int NT, int kMode>
struct Smem {
    using Sh = Shape<D, KIND>;
    // 4-bit rows, 32 requests of up to 4096 keys, 64 of up to 8192, 8 of 16k-32k (us): three
    // blocks and two tiles of 32 keys on their way 21.1, 48.3, 72.2, one 16.4, 47.0, 70.2;
    // two blocks and two tiles 17.5, 53.1, 79.7; four 23.4, 58.5, 76.0; three blocks and one
    // tile of 64 keys 18.3, 50.1, 67.5.
    // Behind a prefix, whose kernel leaves the SMs one by one and whose merge follows: 8
    // bf16 requests, 32 of them, 64 e4m3 requests with two blocks of two tiles 16.4, 37.6,
    // 72.3; three of two 15.8, 38.2, 76.7; three of one 15.7, 36.8, 68.7; four of one 16.9,
    // 39.4, 70.1; two of three 16.3, 38.3, 75.2.
    static constexpr int kStages = KIND == kQ4Pool || (kMode == kSuffix && NT == 1) ? 1 : 2;  // tiles on their way
    static constexpr int kBlocksPerSM = kStages == 1 && NT == 1 ? 3 : 2;
    static constexpr int kSlab = (D / 16 * NT * 4 + 4 * NT) * 32 * 4; // one warp's state: O^T, m, l
    static constexpr int kRing = 0;                                   // [warp][stage][K, V]
    static constexpr int kSlabs = kRing + kWarps * kStages * 2 * Sh::kTileBytes;
    static constexpr int kBars = kSlabs + 2 * kSlab;                  // [warp][stage][K, V]
    static constexpr int kMisc = kBars + kWarps * kStages * 2 * 8;
    // [B + 1] granules before, [B] granules, [B] lengths; kSuffix: [B] firsts, the prefixes'
    // starts and lengths
    static constexpr int kPrefix = kMisc + 16;
    static size_t bytes(int B)
    {
        return kPrefix + size_t(kMode == kSuffix ? 4 * B + 1 + 2 * kMaxPrefixes + 1 : 3 * B + 1) * 4 + 1024;
    }
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
// Behind a shared prefix (kSuffix) the keys from `first` on, of which the tiles
// before the box that holds it are left out; none where the prefix is all.
struct TileSpan {
    int sink_tiles, start, first_seen, granules;
};
template <int kTok, int kMode>
__device__ __forceinline__ TileSpan tile_span(const DecodeArgs& a, int n, int first)
{
    TileSpan s{0, 0, 0, 0};
    if constexpr (kMode == kSuffix) {
        s.first_seen = first;
        s.start = first < n ? first & ~(a.box_rows - 1) : n;
    }
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

// What lies at p, behind a prefix past the first cache (see the kernel's start).
template <int kMode, typename T>
__device__ __forceinline__ T now(const T* p)
{
    return kMode == kSuffix ? __ldcg(p) : *p;
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
    // The output rows of (request, KV head) bh, `rows` of them from q_row0 on: each
    // lane holds runs of neighbouring elements of D.
    template <int KIND, int kMode>
    __device__ __forceinline__ void write(const DecodeArgs& a, int64_t bh, int64_t q_row0, int rows, int lane) const
    {
        constexpr bool F8 = KIND != kBf16Pool;
        const int g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = 8 * nt + 2 * q + rr;
                if (r >= rows)
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
    // The state as rows (unnormalised O [8 NT][D], then (m, l) of each row), the
    // first `rows` of them.
    template <int KIND>
    __device__ __forceinline__ void put_rows(float* to, int rows, int lane) const
    {
        constexpr bool F8 = KIND != kBf16Pool;
        const int g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = 8 * nt + 2 * q + rr;
                if (r >= rows)
                    continue;
                float* dst = to + r * D;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int k = 2 * half + rr;
                    float* run = dst + (D == 64 ? 8 * g + 4 * half : F8 ? 16 * g + 8 * half : 64 * half + 8 * g);
#pragma unroll
                    for (int t = 0; t < kKS; t += 4)
                        *reinterpret_cast<float4*>(run + t) =
                            make_float4(o[t][nt][k], o[t + 1][nt][k], o[t + 2][nt][k], o[t + 3][nt][k]);
                }
                if (g == 0)
                    *reinterpret_cast<float2*>(to + 8 * NT * D + 2 * r) = make_float2(m[nt][rr], l[nt][rr]);
            }
    }
};

// A 4-bit group's step as the multiply-adds that turn codes into f16 take it: bits 0-3 of
// a half of w behind 0x6400 are 1024 + c, bits 4-7 behind 0x5400 are 64 + c, so
//   s (1024 + c) - 1024 s  and  s (64 + c) - 64 s
// are s c, rounded once (-1024 s is an f16: s is at most 60).
struct Q4Step {
    uint32_t s, c, c64;           // f16x2
    __device__ __forceinline__ explicit Q4Step(uint32_t step)
    {
        s = step;
        c = mul_f16x2(step, 0xe400e400u);      // -1024
        c64 = mul_f16x2(step, 0xd400d400u);    // -64
    }
    // The codes in bits 0-3 / 4-7 of both halves of w.
    __device__ __forceinline__ uint32_t low(uint32_t w) const
    {
        return fma_f16x2((w & 0x000f000fu) | 0x64006400u, s, c);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w) const
    {
        return fma_f16x2((w & 0x00f000f0u) | 0x54005400u, s, c64);
    }
};

template <int D, int KIND, int NT, int kMode>
__global__ void __launch_bounds__(kThreads, (Smem<D, KIND, NT, kMode>::kBlocksPerSM))
    decode_rows_kernel(const __grid_constant__ CUtensorMap key_map,
                       const __grid_constant__ CUtensorMap value_map, const DecodeArgs a)
{
    constexpr bool F8 = KIND == kE4m3Pool, Q4 = KIND == kQ4Pool, kP16 = F8 || Q4;
    using Sh = Shape<D, KIND>;
    using Lay = Smem<D, KIND, NT, kMode>;
    constexpr int kStages = Lay::kStages, kTileBytes = Sh::kTileBytes;
    constexpr int kTok = Sh::kTok, kSub = Sh::kSub, kKL = Sh::kKLoads, kVL = Sh::kVLoads, kKS = Sh::kSteps;
    // floats of a piece's state
    constexpr int kSlot = kMode == kSuffix ? suffix_slot_floats(D, NT) : Lay::kSlab / 4;
    // Modes that take more than 16 rows cut them into segments of 16.
    constexpr bool kCut = kMode == kFull || kMode == kSuffix;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int* misc = reinterpret_cast<volatile int*>(smem + Lay::kMisc);
    int32_t* pre = reinterpret_cast<int32_t*>(smem + Lay::kPrefix);
    int32_t* gbr = pre + a.B + 1;
    int32_t* len = gbr + a.B;
    int32_t* firsts = len + a.B;                      // kSuffix
    int32_t* prefix_starts = firsts + a.B;
    int32_t* prefix_lens = prefix_starts + kMaxPrefixes + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int MS = kCut ? a.MS : 1;
    const int per_req = a.H_kv * MS;
    const int cap = context_cap<kMode>(a);
    const float c = a.scale_log2;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBars) + warp * kStages * 2;
    if (lane == 0) {
        for (int i = 0; i < kStages * 2; ++i)
            mbar_init(&bars[i], 1);
        if (warp == 0) {
            misc[0] = 0;                              // a wait ran out
            if constexpr (!Q4) {                      // (4-bit rows come without maps)
                prefetch_tensormap(&key_map);
                prefetch_tensormap(&value_map);
            }
        }
        fence_barrier_init();
    }
    // Behind a prefix the kernel before this one in the stream is the prefix's, of
    // which nothing is read here; the wait for it is at the end. What this kernel reads
    // was written before that one, each of whose blocks lets this one start only after
    // its own wait: by then every write before it has been performed in the device's memory.
    // It is read from there: lengths, tables and queries by loads that pass the first
    // cache by, which may hold older lines (`now`), K and V by TMA. (With the wait here
    // instead, us: 8 requests behind 2048 keys 20.3 for 15.1, 32 behind 16384 35.5 for
    // 32.4, 64 e4m3 requests 64.2 for 56.1.)
    if constexpr (kMode != kSuffix)
        grid_dependency_wait();
    grid_launch_dependents();

    // ---- this block's granules [x_begin, x_end) -------------------------------
    // (A thread a request: one warp, with the prefixes' tables in global memory, took 1 to 2
    // us more.)
    int n = int(threadIdx.x) < a.B ? now<kMode>(a.context_lens + threadIdx.x) : 0;
    if constexpr (kMode == kSuffix) {
#pragma unroll 1
        for (int p = threadIdx.x; p <= a.prefix.count; p += kThreads) {
            prefix_starts[p] = __ldcg(a.prefix.starts + p);
            if (p < a.prefix.count)
                prefix_lens[p] = prefix_len(a.prefix, p);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
        if (b >= kThreads)
            n = now<kMode>(a.context_lens + b);
        n = clamp_context(n, cap, a.err);
        int first = 0;
        if constexpr (kMode == kSuffix) {
            const int p = prefix_of(prefix_starts, a.prefix.count, b);
            firsts[b] = first = p < 0 ? 0 : min(prefix_lens[p], n);
        }
        gbr[b] = tile_span<kTok, kMode>(a, n, first).granules;
        len[b] = n;
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        if (lane == 0)
            pre[0] = 0;
#pragma unroll 1
        for (int base = 0; base < a.B; base += 32) {
            const int b = base + lane;
            int incl = b < a.B ? gbr[b] * per_req : 0;
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
    const int64_t grid = kMode == kSuffix ? suffix_blocks(units, int(gridDim.x))
                                          : int64_t(gridDim.x) < units ? int64_t(gridDim.x) : units;
    const int64_t cta = blockIdx.x;
    if (cta >= grid) {
        if constexpr (kMode == kSuffix)
            grid_dependency_wait();
        return;
    }
    StreamPoint p0, p1;
    granules_at_units(pre, gbr, a.B, per_req, udiv64(cta * units, grid), udiv64((cta + 1) * units, grid),
                      units, kPieceUnits, p0, p1);
    if (p0.x >= p1.x) {
        if constexpr (kMode == kSuffix)
            grid_dependency_wait();
        return;
    }
    // A place in the stream, with what its segment needs: the loads run ahead of
    // the products, across the ends of pieces.
    struct Place {
        SegmentPos sp;
        int in_seg;                       // granule of the segment
        int rest;                         // the block's granules from this one on
        int n;
        TileSpan span;
    };
    auto enter = [&](Place& p) {
        p.n = len[p.sp.b];
        p.span = tile_span<kTok, kMode>(a, p.n, kMode == kSuffix ? firsts[p.sp.b] : 0);
    };
    // First token of the warp's tile of place p, and the end of its run.
    auto tile_at = [&](const Place& p, int* end) {
        const int t = p.in_seg * kWarps + warp;
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
    auto page_of = [&](const Place& p, int t) {
        const int32_t* entry = a.block_table + int64_t(p.sp.b) * a.max_pages + (t >> a.ps_shift);
        return t < 0 ? 0 : kMode == kSuffix ? __ldcg(entry) : __ldg(entry);
    };
    auto row_of = [&](const Place& p, int t, int phys) {
        if (t < 0)
            return -1;
        if (unsigned(phys) >= unsigned(a.num_pages)) {
            atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
            phys = 0;
        }
        return ((phys * a.H_kv + p.sp.h) << a.ps_shift) + (t & ((1 << a.ps_shift) - 1));
    };
    uint8_t* ring = smem + Lay::kRing + warp * (kStages * 2 * kTileBytes);
    constexpr int kHalves = Q4 ? 1 : Sh::kRowBytes / 128;   // 128-byte column blocks of a row
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
            uint8_t* dst = ring + (stage * 2 + v) * kTileBytes + (lane << box_shift) * (Q4 ? Sh::kRowBytes : 128);
            if constexpr (Q4) {
                bulk_load(dst, (v ? a.value_rows : a.key_rows) + int64_t(row) * Sh::kRowBytes,
                          uint32_t(a.box_rows) * Sh::kRowBytes, bar, policy);
            } else {
#pragma unroll
                for (int hf = 0; hf < kHalves; ++hf)
                    tma_load_2d(dst + hf * kHalfBytes, v ? &value_map : &key_map, hf * 64, row, bar, policy);
            }
        }
    };
    // The next tile to be requested, and its rows (found a step ahead).
    Place ahead;
    ahead.sp = segment_at(pre, gbr, per_req, MS, p0.b, p0.hm);
    ahead.in_seg = int(p0.x - ahead.sp.seg_start);
    ahead.rest = int(p1.x - p0.x);
    enter(ahead);
    Place at = ahead;                     // the tile at hand
    auto step = [&](Place& p) {
        if (--p.rest > 0 && ++p.in_seg == p.sp.seg_len) {
            p.sp = next_segment(pre, gbr, per_req, MS, p.sp);
            p.in_seg = 0;
            enter(p);
        }
    };
    int tok = box_token(ahead);                      // the lane's box of the next tile, and its page
    int page = page_of(ahead, tok);
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
        if (ahead.rest > 0) {
            const int row = row_of(ahead, tok, page);
            step(ahead);
            if (ahead.rest > 0) {
                tok = box_token(ahead);
                page = page_of(ahead, tok);
            }
            copy(row, st, 0);
            copy(row, st, 1);
        }
    }
    const int swz = a.swz;                           // 7: swizzled; 0: boxes of fewer than 8 rows
    int stage = 0;
    uint32_t phase = 0;

    while (at.rest > 0) {
        const SegmentPos sp = at.sp;
        const int n = at.n;
        const TileSpan span = at.span;
        const int len_here = min(at.rest, sp.seg_len - at.in_seg);
        const bool opens = at.in_seg == 0, closes = at.in_seg + len_here == sp.seg_len;
        at.rest -= len_here;
        const int row0 = kCut ? sp.ms * kSegmentRows : 0;     // the segment's rows of the R
        const int rows = a.R - row0;                          // (8 NT of them at most)
        const int64_t q_row0 = (int64_t(sp.b) * a.H_q + sp.h * a.G) * a.L + row0;

        // Query fragments: column n = 8 nt + g of Q^T, the elements of D that
        // this lane's K words hold.
        uint32_t qb[NT][kKS][2];
        uint32_t q_sum[NT];                           // 4-bit pools: the group's sum / 32, in two f16
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + (q_row0 + r) * D);
            if constexpr (Q4) {
                // elements 32 q + 8 i + e of the row, e and e + 4 in one register
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (r < rows)
                        w = now<kMode>(reinterpret_cast<const uint4*>(src + 64 * q + 16 * i));
                    const uint32_t x = bf16x2_to_f16x2(w.x), y = bf16x2_to_f16x2(w.y);
                    const uint32_t z = bf16x2_to_f16x2(w.z), u = bf16x2_to_f16x2(w.w);
                    qb[nt][2 * i][0] = __byte_perm(x, z, 0x5410);
                    qb[nt][2 * i][1] = __byte_perm(x, z, 0x7632);
                    qb[nt][2 * i + 1][0] = __byte_perm(y, u, 0x5410);
                    qb[nt][2 * i + 1][1] = __byte_perm(y, u, 0x7632);
                    sum += (f16_sum(x) + f16_sum(y)) + (f16_sum(z) + f16_sum(u));
                }
                sum *= 1.f / kQ4Group;                // within f16's range like the elements
                const float hi = __half2float(__float2half_rn(sum));
                q_sum[nt] = pack_f16x2(hi, sum - hi);
            } else if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (r < rows) {
                        w[0] = now<kMode>(reinterpret_cast<const uint4*>(src + 128 * j + 32 * q));
                        w[1] = now<kMode>(reinterpret_cast<const uint4*>(src + 128 * j + 32 * q + 16));
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
                    if (r < rows)
                        w = now<kMode>(reinterpret_cast<const uint4*>(src + 64 * j + 16 * q));
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
                const int i = r < rows ? (row0 + r) % a.L : a.L - 1;
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
        // 4-bit pools: sum of P times the least value of the lane's group (rows 2 q + rr)
        float om[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            om[nt][0] = om[nt][1] = om[nt][2] = om[nt][3] = 0.f;

        for (const int end_here = at.in_seg + len_here; at.in_seg < end_here; ++at.in_seg) {
            int end;
            const int t0 = tile_at(at, &end);
            const bool busy = t0 < end;              // the last granule may hold fewer than four tiles
            const bool first_run =
                kMode == kWindow && at.in_seg * kWarps + warp < span.sink_tiles;
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
                for (int s = 0; s < kSub && Q4; ++s) {
                    // lane (g, q): group q of keys g and g + 8; the products of a k-step
                    // are those of elements 8 i + 2 j + {0, 4} and {1, 5} of each group
                    uint4 kr[2];
                    uint32_t par[2];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint8_t* at_row = kt + (16 * s + 8 * hh + g) * kQ4RowBytes;
                        kr[hh] = *reinterpret_cast<const uint4*>(at_row + 16 * q);
                        par[hh] = *reinterpret_cast<const uint32_t*>(at_row + kQ4CodeBytes + 4 * q);
                    }
                    const Q4Step s0(__byte_perm(par[0], 0, 0x1010)), s1(__byte_perm(par[1], 0, 0x1010));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w0 = word(kr[0], i) >> (8 * j), w1 = word(kr[1], i) >> (8 * j);
                            const uint32_t A[4] = {s0.low(w0), s1.low(w1), s0.high(w0), s1.high(w1)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16_16816(j ? odd[s][nt] : sc[s][nt], A, qb[nt][2 * i + j][0],
                                              qb[nt][2 * i + j][1]);
                        }
                    // the least values, times 32, with the query's sums over 32
                    const uint32_t A[4] = {mul_f16x2(__byte_perm(par[0], 0, 0x3232), 0x50005000u),
                                           mul_f16x2(__byte_perm(par[1], 0, 0x3232), 0x50005000u), 0u, 0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(sc[s][nt], A, q_sum[nt], 0u);
                }
#pragma unroll
                for (int s = 0; s < kSub && !Q4; ++s) {
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
            const bool more = ahead.rest > 0;
            if (more) {
                row_v = row_of(ahead, tok, page);
                __syncwarp();                        // every lane has read the place
                copy(row_v, stage, 0);
                step(ahead);
                if (ahead.rest > 0) {
                    tok = box_token(ahead);
                    page = page_of(ahead, tok);
                }
            }
            const bool edge = t0 + kTok - 1 > lim_min || t0 + kTok > end || (kMode == kWindow && t0 < low_max) ||
                              (kMode == kSuffix && t0 < span.first_seen);
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
                                if constexpr (kMode == kSuffix)
                                    seen = seen && tok >= span.first_seen;
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
                                if constexpr (Q4)
                                    om[nt][rr] *= f;
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
                            if constexpr (kP16) {
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
                for (int s = 0; s < kSub && Q4; ++s) {
                    // lane (g, q): elements 16 g .. 16 g + 15 of keys 2 q, 2 q + 1 (+ 8)
                    uint2 vr[4];
                    uint32_t par[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 16 * s + 2 * q + (k & 1) + 8 * (k >> 1);
                        vr[k] = *reinterpret_cast<const uint2*>(vt + r * kQ4RowBytes + 8 * g);
                        par[k] = *reinterpret_cast<const uint32_t*>(vt + r * kQ4RowBytes + kQ4CodeBytes + 4 * (g >> 1));
                    }
                    if (edge) {
                        // Keys that no row sees: zeros, whatever the page holds.
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tok = t0 + 16 * s + 2 * q + (k & 1) + 8 * (k >> 1);
                            if (tok >= end || (kMode == kSuffix && tok < span.first_seen)) {
                                vr[k] = make_uint2(0, 0);
                                par[k] = 0;
                            }
                        }
                    }
                    const Q4Step step[2] = {Q4Step(__byte_perm(par[0], par[1], 0x5410)),
                                            Q4Step(__byte_perm(par[2], par[3], 0x5410))};
                    {
                        const uint32_t A[4] = {__byte_perm(par[0], par[1], 0x7632), 0u,
                                               __byte_perm(par[2], par[3], 0x7632), 0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(om[nt], A, ph[s][nt][0], ph[s][nt][1]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {     // elements 2 e, 2 e + 1 of a word
                        uint32_t f[2][2][2];          // [keys 2 q / 2 q + 8][word][element]
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t x0 = j ? vr[2 * kk].y : vr[2 * kk].x;
                                const uint32_t x1 = j ? vr[2 * kk + 1].y : vr[2 * kk + 1].x;
                                const uint32_t x = __byte_perm(x0, x1, e < 2 ? 0x5410 : 0x7632) >> (8 * (e & 1));
                                f[kk][j][0] = step[kk].low(x);
                                f[kk][j][1] = step[kk].high(x);
                            }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t A[4] = {f[0][0][u], f[0][1][u], f[1][0][u], f[1][1][u]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16_16816(o[2 * e + u][nt], A, ph[s][nt][0], ph[s][nt][1]);
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < kSub && !Q4; ++s) {
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
                            if (tok >= end || (kMode == kWindow && tok >= a.sinks && tok < span.first_seen) ||
                                (kMode == kSuffix && tok < span.first_seen))
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
        if constexpr (Q4) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < kKS; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[t][nt][k] += om[nt][k & 1];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][rr] += __shfl_xor_sync(0xffffffffu, l[nt][rr], off);
        __syncthreads();                             // the piece before has read the slabs
        st.gather(reinterpret_cast<float*>(smem + Lay::kSlabs), warp, lane);
        if (warp == 0 && (kMode == kSuffix || !misc[0])) {
            if constexpr (kMode == kSuffix) {
                // (after a wait that ran out too: what follows finds its places by these notes)
                st.template put_rows<KIND>(a.partials + (int64_t(sp.seg) + cta) * kSlot, rows, lane);
                if (lane == 0) {
                    if (opens)
                        a.note_segment[sp.seg].x = int(cta);
                    if (closes)
                        a.note_segment[sp.seg].y = int(cta);
                }
            } else if (opens && closes)
                st.template write<KIND, kMode>(a, int64_t(sp.b) * a.H_kv + sp.h, q_row0, rows, lane);
            else                                     // a slot of its own: segment and block
                st.put(a.partials + (int64_t(sp.seg) + cta) * kSlot, lane);
        }
        // on to the next segment
        if (at.rest > 0) {
            at.sp = next_segment(pre, gbr, per_req, MS, sp);
            at.in_seg = 0;
            enter(at);
        }
    }
    // What follows reads the prefix's states too.
    if constexpr (kMode == kSuffix)
        grid_dependency_wait();
}

// The segments that straddle blocks: one block each (the others return once the
// first kernel is done). Warp w folds pieces w, w + 4, ... in order, one on its
// way while the one before is folded in.
template <int D, int KIND, int NT, int kMode>
__global__ void __launch_bounds__(kThreads) decode_rows_merge_kernel(const DecodeArgs a, int decode_grid)
{
    using Sh = Shape<D, KIND>;
    using State = RowState<D, NT>;
    constexpr int kSlot = State::kPlaces * 32;
    __shared__ float slabs[2 * kSlot];
    __shared__ int red[2][kWarps];
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seg = blockIdx.x;
    const int MS = kMode == kFull ? a.MS : 1;
    const int per_req = a.H_kv * MS;
    const int b = seg / per_req, hm = seg - b * per_req;
    const int h = MS == 1 ? hm : hm / MS, row0 = (hm - h * MS) * kSegmentRows;
    const int cap = context_cap<kMode>(a);
    auto granules = [&](int r) {
        const int n = __ldcg(a.context_lens + r);
        return tile_span<Sh::kTok, kMode>(a, n < 0 ? 0 : n > cap ? cap : n, 0).granules;
    };
    // The split of the first kernel, from its inputs (which were complete before
    // it let this one start).
    int before = 0, total = 0;
#pragma unroll 1
    for (int r = threadIdx.x; r < a.B; r += kThreads) {
        const int gs = granules(r) * per_req;
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
    const int64_t units = total + int64_t(kPieceUnits) * a.B * per_req;
    const int64_t grid = int64_t(decode_grid) < units ? int64_t(decode_grid) : units;
    const int64_t u0 = before + int64_t(hm) * len + int64_t(kPieceUnits) * (seg + 1);
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
        st.template write<KIND, kMode>(a, int64_t(b) * a.H_kv + h, (int64_t(b) * a.H_q + h * a.G) * a.L + row0,
                                       a.R - row0, lane);
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, DecodeArgs);
using Merge = void (*)(DecodeArgs, int);
struct Kernels {
    Kernel main;
    Merge merge;                  // kSuffix: none
};
// Each in a translation unit of its own.
Kernels q4_kernels(int NT);
Kernels suffix_kernels(int D, int kind, int NT);

template <int D, int KIND, int NT, int kMode>
Kernels kernels_of()
{
    if constexpr (kMode == kSuffix)
        return {decode_rows_kernel<D, KIND, NT, kMode>, nullptr};
    else
        return {decode_rows_kernel<D, KIND, NT, kMode>, decode_rows_merge_kernel<D, KIND, NT, kMode>};
}

}  // namespace rows
}  // namespace pa

