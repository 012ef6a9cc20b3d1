// Decode of a batch whose requests share prefixes, first and last step.
//
// The rows of all requests that share a prefix attend to it together. With the prefix's
// keys j = 0 .. N - 1 and any row r of one of its requests,
//   s_rj = c q_r . k_j,  m_r = max s,  l_r = sum 2^(s - m),  O_r = sum 2^(s - m) v_j
// over the keys the row sees (log2 domain, c = scale log2 e). The G L rows that a
// request has for a KV head, one request behind the other, are the 128-row tiles
// of tcgen05 products: K and V are read once for 256 rows (where a decode over each
// request's own table reads them once a request). The few-row kernel behind this one
// does the requests' own keys, and the merge kernel here joins the states of a row:
//   M = max m,  out = sum O 2^(m - M) / sum l 2^(m - M).
//
// An item is (prefix, KV head, block of 256 rows), a unit of work a tile of 128 keys. The
// tiles of all items form one stream that the grid cuts into equal ranges; every range
// leaves a state of its own for each item it touches (slot: item + block, distinct
// because both ascend), so no block waits for another.
//
// A block has two softmax warpgroups. With more than 128 rows each holds 128 of them and
// both take every tile; with up to 128 both hold the same rows and take the tiles in
// turn (two states a slot). Either way the products are a chain of steps that alternate
// between the warpgroups:
//   S(j) = Q K^T,  softmax (lazy rescale at 2^8),  O += P V(j),  S(j + 2) over P(j).
//
//   * bf16 pools, warp 0: K tiles, warp 2: V tiles by TMA, page by page, two stages each;
//   * e4m3 and 4-bit pools, warp 0: tiles of codes by TMA into a ring, warps 12-15: codes
//     into f16 (K two stages, V one); Q and P are f16 then. (A copy of the prefixes as
//     bf16 pages before this kernel took 42 of 107 us for 64 e4m3 requests over 31000
//     shared keys; three converting warps that asked for their codes themselves took 2.3
//     us a tile, register loads 4.);
//   * warp 1 (one elected thread): the tcgen05.mma chain;
//   * warps 4-7 and 8-11: the query rows of a piece into shared memory, the softmax
//     (P over the upper half of the scores' columns in TMEM, rounded to bf16: its error,
//     2^-9 of a term, averages out below the output's own rounding), the states.
// TMEM (512 columns): S_0, S_1, O_0, O_1 (128 each).
//
// Measured, a call (three kernels), and the plain decode over tables that name the same
// pages, which then lie in L2: 8 bf16 requests behind 2048 keys 14.8 us, plain 14.1; 32 in
// groups of 7 behind 16384 keys 32.3 (57 MB), 134; 64 e4m3 requests behind 3 prefixes, 31000
// keys in all, 56 (140 MB), 225; 16 chunks of 4 rows behind 8192 4-bit keys 39.5, 70. The
// plain call is ahead up to about 16000 shared positions of all requests together, this one
// from about 32000. What bounds it: a chain of three kernels, 2 us from one to the next, and
// in each what a block does once (about 2 us to its pieces, 2 to its rows, 1.5 for the
// first run of its instructions, 2 to write a state); the states themselves (20 MB written
// and read again with 38 blocks an item); from about ten tiles a block on the steps: 1.25
// us a tile of 2 x 128 rows, and with codes 1.4 for one of 128, most of it their
// conversion.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefix.cuh"
#include "pa_q4.cuh"
#include "pa_split.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kKeys = 128;            // keys per tile
constexpr int kMaxPieces = kPrefixMaxPieces;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;

__host__ __device__ constexpr uint32_t col_s(int half) { return uint32_t(half * 128); }
__host__ __device__ constexpr uint32_t col_o(int half) { return uint32_t(256 + half * 128); }
constexpr uint32_t kPCol = 64;

// Pools of codes: each of four warps turns kRunKeys keys of every K and V tile into f16;
// kRing tiles of codes are on their way to them.
constexpr int kRunKeys = 32, kConverters = kKeys / kRunKeys, kRing = 3;

template <int D, int KIND>
struct Layout {
    static constexpr bool kCodes = KIND != kBf16Pool;
    static constexpr int kVStages = kCodes ? 1 : 2;     // the ring takes the second one's place
    static constexpr int kRowBytes = KIND == kQ4Pool ? kQ4RowBytes : D;   // of codes
    static constexpr int kCodeTile = kKeys * kRowBytes;
    static constexpr int kThreads = kCodes ? 512 : 384;
    // Registers a thread: warps 0-3, the two softmax warpgroups, the converters.
    static constexpr int kRegsFirst = kCodes ? 64 : 128;
    static constexpr int kRegsSoftmax = kCodes ? 176 : 184;
    static constexpr int kRegsConvert = kCodes ? 88 : 0;
    static constexpr int kRegsSum = 128 * (kRegsFirst + 2 * kRegsSoftmax + kRegsConvert);
    static_assert(kRegsSum <= 65536, "register split");
    static constexpr int kBlock = 128 * 128;            // 128 rows x 64 elements (128 B)
    static constexpr int kMat = D / 64 * kBlock;        // 128 x D, [column block][row][128 B]
    static constexpr int kQ = 0;                        // [half]
    static constexpr int kK = kQ + 2 * kMat;            // 2 stages
    static constexpr int kV = kK + 2 * kMat;
    static constexpr int kCodeRing = kV + kVStages * kMat;   // [slot][key][row bytes]
    static constexpr int kBar = kCodeRing + (kCodes ? kRing * kCodeTile : 0);
    static constexpr int kNumBars = 16 + (kCodes ? 2 * kRing : 1);
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kMisc = kTmemSlot + 16;
    static constexpr int kSlotInfo = kMisc + 16;        // [slot] (tile and matrix, keys)
    static constexpr int kPieces = kSlotInfo + (kCodes ? kRing * 8 : 0);   // Piece[kMaxPieces]
    static constexpr int kGroups = kPieces + kMaxPieces * 36;              // Group[count]
};

// Barrier indices.
constexpr int kQFull = 0;     // + half (2)
constexpr int kKFull = 2;     // + stage (2)
constexpr int kKEmpty = 4;
constexpr int kVFull = 6;
constexpr int kVEmpty = 8;
constexpr int kSFull = 10;    // + half (2)
constexpr int kPFull = 12;    // + half
constexpr int kPVDone = 14;   // + half
constexpr int kFirstKeys = 16;   // bf16 pools: arrived at once
constexpr int kCodeFull = 16; // + slot (kRing)
constexpr int kCodeEmpty = kCodeFull + kRing;

// A tile weighs kTileUnits, an item kItemUnits more (its rows, its state); a tile belongs to
// the block whose range holds its first unit. A block has at least kLeastUnits (but the
// last), so that no range lies inside a tile. 64 e4m3 requests behind 3 prefixes, 16
// chunks of 4 over 4-bit pages (us): an item 4 units 58.1, 41.9; 8 57.4, 39.8; 16 56.2,
// 39.6. 8 requests behind 2048 keys: at least 8 units 14.7, 12 15.4, 16 16.2.
constexpr int kTileUnits = 4;
constexpr int kItemUnits = 16;
constexpr int kLeastUnits = 8;

// One prefix: its keys, its first request, its rows for one KV head; where its units and
// items start in the stream.
struct Group {
    int len, first, rows, items, us, item;
    __device__ __forceinline__ int tiles() const { return (len + kKeys - 1) / kKeys; }
    __device__ __forceinline__ int item_units() const { return tiles() * kTileUnits + kItemUnits; }
    __device__ __forceinline__ int units() const { return items * item_units(); }
};

// *bad: the starts do not ascend within the batch.
__device__ __forceinline__ Group group_at(const PrefixKernelArgs& a, int p, bool* bad)
{
    Group g;
    g.first = __ldg(a.prefix.starts + p);
    const int end = __ldg(a.prefix.starts + p + 1);
    *bad = g.first < 0 || end < g.first || end > a.B;
    g.len = prefix_len(a.prefix, p);
    g.rows = *bad ? 0 : (end - g.first) * a.R;
    g.items = g.len > 0 ? a.H_kv * ((g.rows + 255) / 256) : 0;
    g.us = g.item = 0;
    return g;
}

// The ranges of U units that G blocks take: U / G each, the first U % G one more.
struct Ranges {
    int G, per, rem;
    __device__ __forceinline__ Ranges(int U, int grid)
    {
        G = max(1, min(grid, U / kLeastUnits));
        per = U / G;
        rem = U - per * G;
    }
    __device__ __forceinline__ int start(int c) const { return c * per + min(c, rem); }
    __device__ __forceinline__ int of(int u) const       // the block whose range holds unit u
    {
        const int longer = rem * (per + 1);
        return u < longer ? u / (per + 1) : rem + (u - longer) / per;
    }
};

// The part of an item in a block's range of units.
struct Piece {
    int p, len, k0, k1;      // prefix, its keys; tiles
    int h, rb, rows, first;  // KV head, block of 256 rows; the prefix's rows and first request
    int item;                // of all
};

// A block's pieces: the first kMaxPieces in shared memory, what there may be more (many
// short prefixes beside a long one) in the workspace.
struct Pieces {
    Piece* near;
    Piece* far;
    __device__ __forceinline__ Piece& operator[](int i) const
    {
        return *(i < kMaxPieces ? near + i : far + (i - kMaxPieces));
    }
};

// The first tile of an item (first unit us) that starts at or after unit x.
__device__ __forceinline__ int tile_at(int x, int us, int tiles)
{
    const int d = x - us - kItemUnits;
    return d <= 0 ? 0 : min(tiles, (d + kTileUnits - 1) / kTileUnits);
}

// The products' steps, in order: a step is one warpgroup's (half's) work on one tile.
// Half j & 1 takes step j; `first` / `last` of its piece for that half, `opens` /
// `closes` the tile's loads.
struct Step {
    int g;                   // tile of the block's stream
    bool first, opens, closes, valid;
};
struct StepIter {
    int i, k, k1, g;              // next piece; next tile of this one, its end, of the stream
    int sub, done;                // steps of the tile, of the piece
    bool pair;
    __device__ __forceinline__ Step next(const Pieces& pieces, int count)
    {
        Step st;
        st.valid = false;
        if (k >= k1) {
            if (i >= count)
                return st;
            k = pieces[i].k0;
            k1 = pieces[i].k1;
            pair = pieces[i].rows > 128;
            sub = done = 0;
            ++i;
        }
        st.valid = true;
        st.g = g;
        st.first = done < 2;
        st.opens = sub == 0;
        st.closes = !pair || sub == 1;
        ++done;
        if (st.closes) {
            sub = 0;
            ++k;
            ++g;
        } else {
            ++sub;
        }
        return st;
    }
};

// A run's codes at `from` as f16 into a [column block][key][128 bytes] matrix, swizzled; the
// first `live` keys of it, zeros behind them. Of every 8 elements of 4-bit rows the order
// is 0 4 1 5 2 6 3 7, as their codes come apart: Q has it too, and the states are put
// right as they are written.
// kEnds: fewer than kRunKeys of them.
template <int KIND, bool kEnds>
__device__ __forceinline__ void convert_run(uint8_t* mat, int block_bytes, const uint8_t* from, int key0, int live,
                                            int lane)
{
    constexpr bool kQ4 = KIND == kQ4Pool;
    constexpr int kRowBytes = kQ4 ? kQ4RowBytes : 128;
    constexpr int kChunks = kQ4 ? 4 : 8;                         // 16-byte pieces of a row's codes
    constexpr int kOut = kQ4 ? 4 : 2;                            // 16-byte pieces of f16 from each
    const int c = lane % kChunks;
    // Lanes whose pieces go to the second column block take another key's: the eight lanes
    // of a store then meet eight different bank groups.
    const int turn = c >= kChunks / 2 ? kOut / 2 : 0;
    // Half of them at a time, all read before the first is stored. (All at once: 1 us more a
    // call. Instructions that a block runs for the first time cost it about 5 cycles each.)
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        uint4 codes[kChunks / 2];
        uint32_t params[kQ4 ? kChunks / 2 : 1];
        const int row0 = half * 16 + lane / kChunks;
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i) {
            const uint8_t* row = from + ((row0 + i * (32 / kChunks)) ^ turn) * kRowBytes;
            codes[i] = *(reinterpret_cast<const uint4*>(row) + c);
            if constexpr (kQ4)
                params[i] = *(reinterpret_cast<const uint32_t*>(row + kQ4CodeBytes) + c);
        }
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i) {
            const int r = (row0 + i * (32 / kChunks)) ^ turn;
            const uint4 x = codes[i];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t v[4 * kOut];
            if constexpr (kQ4) {
                const uint32_t s = __byte_perm(params[i], 0, 0x1010), m = __byte_perm(params[i], 0, 0x3232);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // c exactly (1024 + c - 1024, 64 + c - 64), then m + s c
                        const uint32_t y = w[k] >> (8 * j);
                        const uint32_t lo = add_f16x2((y & 0x000f000fu) | 0x64006400u, 0xe400e400u);
                        const uint32_t hi = add_f16x2((y & 0x00f000f0u) | 0x54005400u, 0xd400d400u);
                        v[4 * k + 2 * j] = fma_f16x2(lo, s, m);
                        v[4 * k + 2 * j + 1] = fma_f16x2(hi, s, m);
                    }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k] = e4m3x2_to_f16x2(w[k]);
                    v[2 * k + 1] = e4m3x2_hi_to_f16x2(w[k]);
                }
            }
            const int key = key0 + r;
#pragma unroll
            for (int k = 0; k < kOut; ++k) {
                const int ch = c * kOut + k;   // 16-byte piece of the f16 row
                *reinterpret_cast<uint4*>(mat + (ch >> 3) * block_bytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4)) =
                    !kEnds || r < live ? make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3])
                                       : make_uint4(0, 0, 0, 0);
            }
        }
    }
}

// Two f16 pairs of neighbours (elements 2 i, 2 i + 1 of 8) as 4-bit rows have them.
__device__ __forceinline__ uint4 apart(uint4 v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
}

template <int D, int KIND>
__global__ void __launch_bounds__((Layout<D, KIND>::kThreads), 1)
    prefix_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap value_map,
                  const PrefixKernelArgs a)
{
    using Lay = Layout<D, KIND>;
    constexpr int kVStages = Lay::kVStages;
    constexpr bool kCodes = KIND != kBf16Pool;
    constexpr int kBlocks = D / 64;                      // 128-byte column blocks of a row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kTmemSlot);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + Lay::kMisc);
    const Pieces pieces = {reinterpret_cast<Piece*>(smem + Lay::kPieces),
                           static_cast<Piece*>(a.more_pieces) + int64_t(blockIdx.x) * a.most_items};
    static_assert(sizeof(Piece) == 36, "as laid out");
    __shared__ int piece_count, all_units;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        misc[0] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[kQFull + i], 4);              // one arrival per warp
            mbar_init(&bar[kKFull + i], kCodes ? kConverters : 1);
            mbar_init(&bar[kKEmpty + i], 1);
            mbar_init(&bar[kVFull + i], kCodes ? kConverters : 1);
            mbar_init(&bar[kVEmpty + i], 1);
            mbar_init(&bar[kSFull + i], 1);
            mbar_init(&bar[kPFull + i], 4);
            mbar_init(&bar[kPVDone + i], 1);
        }
        for (int i = 0; i < kRing && kCodes; ++i) {
            mbar_init(&bar[kCodeFull + i], 1);
            mbar_init(&bar[kCodeEmpty + i], kConverters);
        }
        if (!kCodes)
            mbar_init(&bar[kFirstKeys], 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    grid_dependency_wait();
    grid_launch_dependents();
    // The queries into L2, before the keys queue up in front of them (a block's rows came
    // in 4 us after they were asked for).
    {
        const int64_t lines = (int64_t(a.B) * a.H_q * a.L * D * 2 + 127) / 128;
#pragma unroll 1
        for (int64_t i = int64_t(blockIdx.x) * Lay::kThreads + threadIdx.x; i < lines;
             i += int64_t(gridDim.x) * Lay::kThreads)
            prefetch_l2(reinterpret_cast<const uint8_t*>(a.q) + i * 128);
    }
    // ---- the prefixes' places in the stream, and this block's pieces ---------------
    const int c = int(blockIdx.x);
    if (warp == 0) {
        Group* groups = reinterpret_cast<Group*>(smem + Lay::kGroups);
        const int prefixes = a.prefix.count;
        int us = 0, item = 0;
        bool bad = false;
#pragma unroll 1
        for (int base = 0; base < prefixes; base += 32) {
            const int p = base + lane;
            Group g;
            g.len = g.items = 0;
            if (p < prefixes) {
                bool no;
                g = group_at(a, p, &no);
                bad |= no;
                if (c == 0) {
                    const int n = __ldg(a.prefix.lens + p);
                    if (n < 0 || n > a.prefix.cap)
                        atomicOr(a.err, PA_DEVERR_CONTEXT_LEN_BIT);
                }
            }
            int incl_u = g.units(), incl_i = g.items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl_u, o), v = __shfl_up_sync(0xffffffffu, incl_i, o);
                if (lane >= o) {
                    incl_u += u;
                    incl_i += v;
                }
            }
            if (p < prefixes) {
                g.us = us + incl_u - g.units();
                g.item = item + incl_i - g.items;
                groups[p] = g;
            }
            us += __shfl_sync(0xffffffffu, incl_u, 31);
            item += __shfl_sync(0xffffffffu, incl_i, 31);
        }
        // Rows counted twice would have more states than there is room for: none then.
        bad = __any_sync(0xffffffffu, bad);
        if (bad && c == 0 && lane == 0)
            atomicOr(a.err, PA_DEVERR_PREFIX_BIT);
        const int U = bad ? 0 : us;
        const Ranges ranges(U, int(gridDim.x));
        int found = 0;
        if (U > 0 && c < ranges.G) {
            const int s = ranges.start(c), e = ranges.start(c + 1);
#pragma unroll 1
            for (int base = 0; base < prefixes; base += 32) {
                const int p = base + lane;
                int i0 = 0, n = 0;
                Group g;
                if (p < prefixes) {
                    g = groups[p];
                    const int w = g.item_units(), end = g.us + g.units();
                    if (g.items > 0 && g.us < e && s < end) {
                        i0 = (max(s, g.us) - g.us) / w;
                        int i1 = (min(e, end) - 1 - g.us) / w;
                        // an item whose tiles all start before the range, or behind it
                        if (tile_at(s, g.us + i0 * w, g.tiles()) == g.tiles())
                            ++i0;
                        if (tile_at(e, g.us + i1 * w, g.tiles()) == 0)
                            --i1;
                        n = max(0, i1 - i0 + 1);
                    }
                }
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o)
                        incl += v;
                }
                const int blocks = n > 0 ? (g.rows + 255) / 256 : 1;
#pragma unroll 1
                for (int x = 0; x < n; ++x) {
                    const int at = found + incl - n + x, i = i0 + x;
                    Piece& pc = pieces[at];
                    const int h = i / blocks;
                    pc.p = p;
                    pc.len = g.len;
                    pc.k0 = tile_at(s, g.us + i * g.item_units(), g.tiles());
                    pc.k1 = tile_at(e, g.us + i * g.item_units(), g.tiles());
                    pc.h = h;
                    pc.rb = i - h * blocks;
                    pc.rows = g.rows;
                    pc.first = g.first;
                    pc.item = g.item + i;
                }
                found += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        if (lane == 0) {
            piece_count = found;
            all_units = U;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int count = piece_count;
    // ---- notes for the merge: where each row's states are (warp 3)
    auto write_notes = [&]() {
        const Group* groups = reinterpret_cast<const Group*>(smem + Lay::kGroups);
        const Ranges ranges(all_units, int(gridDim.x));
        const int rows = a.B * a.H_kv * a.R;
#pragma unroll 1
        for (int row = c * 32 + lane; row < rows; row += int(gridDim.x) * 32) {
            const int bh = a.by_R.of(row), x = row - bh * a.R, b = a.by_H.of(bh), h = bh - b * a.H_kv;
            int4 note = make_int4(0, 0, 0, 0);
            if (all_units > 0 && b >= groups[0].first) {
                int p = 0;                               // the last prefix that starts at b or before
#pragma unroll 1
                for (int hi = a.prefix.count; hi - p > 1;) {
                    const int mid = (p + hi) >> 1;
                    if (groups[mid].first <= b)
                        p = mid;
                    else
                        hi = mid;
                }
                const Group g = groups[p];
                const int f = (b - g.first) * a.R + x;
                if (f < g.rows && g.items > 0) {
                    const int i = h * ((g.rows + 255) >> 8) + (f >> 8);
                    const int u = g.us + i * g.item_units() + kItemUnits;
                    const int from = ranges.of(u), to = ranges.of(u + (g.tiles() - 1) * kTileUnits);
                    const int twice = g.rows > 128 ? 0 : 1;
                    note = make_int4(g.item + i + from, (to - from + 1) << twice, f & 255, twice);
                }
            }
            a.note_row[row] = note;
        }
    };
    if (count == 0) {
        if (warp == 1)
            tmem_dealloc(tmem, kTmemCols);
        if (warp == 3)
            write_notes();
        return;
    }

    const uint32_t sQ = smem_u32(smem + Lay::kQ), sK = smem_u32(smem + Lay::kK), sV = smem_u32(smem + Lay::kV);
    if (warp < 4) {
        setmaxnreg_dec<Lay::kRegsFirst>();
        if (kCodes && warp == 0) {
            // ===================== tiles of codes ====================================
            if constexpr (kCodes) {
                const uint64_t policy = l2_policy_evict_last();  // the item's other row blocks read it too
                const int box = min(a.ps, kKeys);
                const int box_shift = min(a.ps_shift, 7);
                int2* info = reinterpret_cast<int2*>(smem + Lay::kSlotInfo);
                // The order: K of tile 0, then K of tile g + 1 and V of tile g in turn, so that
                // the wait for V's one stage (the product before) keeps no K from the scores
                // ahead.
                struct Tile {                            // tile k of a piece, g of the block's stream
                    int i, k, k1, g;
                };
                auto pass = [&](Tile& t) {
                    ++t.g;
                    if (++t.k >= t.k1 && ++t.i < count) {
                        t.k = pieces[t.i].k0;
                        t.k1 = pieces[t.i].k1;
                    }
                };
                Tile kt = {0, pieces[0].k0, pieces[0].k1, 0};
                Tile vt = kt;
                const uint32_t ps_mask = (1u << a.ps_shift) - 1u;
                int u = 0;                               // tiles of codes asked for
                auto slot_free = [&](int slot) {
                    return mbar_wait_warp(&bar[kCodeEmpty + slot], ((u / kRing) & 1) ^ 1u, misc, a.err);
                };
                struct Pages {                           // of a tile's boxes 32 i + lane
                    int id[kKeys / 32];
                };
                auto lookup = [&](const Tile& t) {
                    Pages pages;
                    const int first = t.k * kKeys;
                    const Piece& pc = pieces[t.i];
                    const int boxes = (min(kKeys, pc.len - first) + box - 1) >> box_shift;
                    const int32_t* table = a.prefix.table + int64_t(pc.p) * a.prefix.pages;
#pragma unroll
                    for (int i = 0; i < kKeys / 32; ++i)
                        pages.id[i] =
                            32 * i + lane < boxes
                                ? __ldg(table + ((first + ((32 * i + lane) << box_shift)) >> a.ps_shift)) : 0;
                    return pages;
                };
                auto request = [&](const Tile& t, bool is_v, const Pages& pages) {
                    const int slot = u % kRing;
                    const int first = t.k * kKeys;
                    const Piece& pc = pieces[t.i];
                    const int live = min(kKeys, pc.len - first);
                    const int boxes = (live + box - 1) >> box_shift;
                    const bool ok = slot_free(slot);
                    if (ok) {
                        if (lane == 0) {
                            info[slot] = make_int2(2 * t.g + (is_v ? 1 : 0), live);
                            mbar_arrive_expect_tx(&bar[kCodeFull + slot], uint32_t(boxes * box * Lay::kRowBytes));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < kKeys / 32; ++i) {
                            const int at = (32 * i + lane) << box_shift;
                            if (32 * i + lane < boxes) {
                                int page = pages.id[i];
                                if (unsigned(page) >= unsigned(a.num_pages)) {
                                    atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
                                    page = 0;
                                }
                                const uint32_t row = (uint32_t(page * a.H_kv + pc.h) << a.ps_shift) +
                                                     (uint32_t(first + at) & ps_mask);
                                bulk_load(smem + Lay::kCodeRing + slot * Lay::kCodeTile + at * Lay::kRowBytes,
                                          (is_v ? a.value_rows : a.key_rows) + uint64_t(row) * Lay::kRowBytes,
                                          uint32_t(box * Lay::kRowBytes), &bar[kCodeFull + slot], policy);
                            }
                        }
                    }
                    __syncwarp();
                    ++u;
                };
                // Pages are looked up a request ahead; V's are those that K had.
                Pages next = lookup(kt), now = next, held = next;
                auto request_k = [&]() {
                    now = next;
                    request(kt, false, now);
                    pass(kt);
                    if (kt.i < count)
                        next = lookup(kt);
                };
                request_k();
                held = now;
                while (vt.i < count) {
                    if (kt.i < count)
                        request_k();
                    request(vt, true, held);
                    pass(vt);
                    held = now;
                }
                // The end, and no copy still landing: the converters have waited for each.
                const int slot = u % kRing;
                slot_free(slot);
                if (lane == 0) {
                    info[slot] = make_int2(-1, 0);
                    mbar_arrive(&bar[kCodeFull + slot]);
                }
#pragma unroll 1
                for (int i = 1; i < kRing; ++i) {
                    ++u;
                    slot_free(u % kRing);
                }
            }
        } else if (!kCodes && (warp == 0 || warp == 2)) {
            // ===================== K (warp 0) and V (warp 2) tiles ===================
            const bool is_v = warp == 2;
            const CUtensorMap* map = is_v ? &value_map : &key_map;
            uint8_t* to = smem + (is_v ? Lay::kV : Lay::kK);
            const int full = is_v ? kVFull : kKFull, empty = is_v ? kVEmpty : kKEmpty;
            const uint64_t policy = l2_policy_evict_last();  // the item's other row blocks read it too
            if (lane == 0)
                prefetch_tensormap(map);
            const int box = a.box_rows;                  // min(page size, 128), at least 8
            // (a tile's pages are looked up while the tile before is waited for)
            auto page_at = [&](int i, int k) {
                const int key0 = k * kKeys + lane * box;
                return lane * box < kKeys && key0 < pieces[i].len
                           ? __ldg(a.prefix.table + int64_t(pieces[i].p) * a.prefix.pages + (key0 >> a.ps_shift)) : 0;
            };
            // The first keys are here before the first values are asked for: every block starts at
            // once, and the scores need the keys (32 requests behind 16384 keys 32.8 -> 32.2 us; the
            // second keys held back too: 32.5). Warp 0 says so, on a barrier that completes
            // once: it refills the keys' stage itself, so it sees that stage's first phase.
            // Warp 2 there could come two phases late, when the parity is the same again,
            // and the keys would wait for products that wait for its values.
            auto first_keys = [&]() {
                mbar_wait_warp(&bar[kKFull], 0, misc, a.err);
                if (lane == 0)
                    mbar_arrive(&bar[kFirstKeys]);
            };
            int g = 0, next = page_at(0, pieces[0].k0);
            for (int i = 0; i < count; ++i) {
                const int n = pieces[i].len, k1 = pieces[i].k1, head = pieces[i].h;
                for (int k = pieces[i].k0; k < k1; ++k, ++g) {
                    const int key0 = k * kKeys;
                    const int boxes = (min(n, key0 + kKeys) - key0 + box - 1) / box;
                    const int tok = key0 + lane * box;
                    int phys = next;
                    if (k + 1 < k1)
                        next = page_at(i, k + 1);
                    else if (i + 1 < count)
                        next = page_at(i + 1, pieces[i + 1].k0);
                    const int st = g & 1;
                    if (is_v && g == 0)
                        mbar_wait_warp(&bar[kFirstKeys], 0, misc, a.err);
                    if (!is_v && g == 2)             // both stages asked for
                        first_keys();
                    const bool ok = mbar_wait_warp(&bar[empty + st], ((g >> 1) & 1) ^ 1u, misc, a.err);
                    if (ok) {
                        if (lane == 0)
                            mbar_arrive_expect_tx(&bar[full + st], uint32_t(boxes) * box * 128u * kBlocks);
                        __syncwarp();
                        if (lane < boxes) {
                            if (unsigned(phys) >= unsigned(a.num_pages)) {
                                atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
                                phys = 0;
                            }
                            const int row = ((phys * a.H_kv + head) << a.ps_shift) + (tok & (a.ps - 1));
                            uint8_t* dst = to + st * Lay::kMat + lane * box * 128;
#pragma unroll
                            for (int x = 0; x < kBlocks; ++x)
                                tma_load_2d(dst + x * Lay::kBlock, map, 64 * x, row, &bar[full + st], policy);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!is_v && g <= 2)
                first_keys();
            // No copy may still be landing when the block exits.
#pragma unroll 1
            for (int i = max(0, g - 2); i < g; ++i)
                mbar_wait_bounded(&bar[full + (i & 1)], (i >> 1) & 1, misc, a.err);
        } else if (warp == 3) {
            // (not before the registers are handed over: the softmax waits for them)
            write_notes();
        } else if (warp == 1) {
            // ===================== MMA issue (one elected thread) =====================
            const bool leader = elect_one();
            const uint32_t idesc_s = kCodes ? idesc_f16_f32(128, kKeys, 0) : idesc_bf16_f32(128, kKeys, 0);
            const uint32_t idesc_pv = kCodes ? idesc_f16_f32(128, D, 1) : idesc_bf16_f32(128, D, 1);
            const uint64_t dq = smem_desc_sw128(sQ, 16u, 1024u), dk = smem_desc_sw128(sK, 16u, 1024u);
            const uint64_t dv = smem_desc_sw128(sV, uint32_t(Lay::kBlock), 1024u);
            auto k_major = [](int kk) { return uint32_t(kk >> 2) * Lay::kBlock + uint32_t(kk & 3) * 32u; };
            auto wait = [&](int bi, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait_lean(&bar[bi], parity, misc, a.err));
            };
            auto commit = [&](int bi) {
                if (leader)
                    tc_commit(&bar[bi]);
                __syncwarp();
            };
            int rounds[2] = {0, 0};                      // query tiles waited for, by half
            auto scores = [&](int j, const Step& st) {
                const int h = j & 1, stage = st.g & 1;
                if (st.first) {
                    if (!wait(kQFull + h, rounds[h] & 1))
                        return false;
                    ++rounds[h];
                }
                if (!wait(kKFull + stage, (st.g >> 1) & 1))
                    return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_bf16(tmem + col_s(h), desc_advance(dq, uint32_t(h * Lay::kMat) + k_major(kk)),
                                    desc_advance(dk, uint32_t(stage * Lay::kMat) + k_major(kk)), idesc_s, kk > 0);
                }
                __syncwarp();
                commit(kSFull + h);
                if (st.closes)
                    commit(kKEmpty + stage);
                return true;
            };
            StepIter it;
            it.i = it.k = it.k1 = it.g = 0;
            Step now = it.next(pieces, count), next = it.next(pieces, count);
            bool ok = now.valid && scores(0, now) && (!next.valid || scores(1, next));
            int j = 0;
            for (; ok && now.valid; ++j) {
                const int h = j & 1, stage = kVStages == 1 ? 0 : now.g & 1;
                const uint32_t phase = (j >> 1) & 1;
                if (!wait(kPFull + h, phase) || !wait(kVFull + stage, (kVStages == 1 ? now.g : now.g >> 1) & 1))
                    break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc_mma_bf16_ts(tmem + col_o(h), tmem + col_s(h) + kPCol + 8u * kk,
                                       desc_advance(dv, uint32_t(stage * Lay::kMat) + uint32_t(kk) * 16u * 128u),
                                       idesc_pv, (!now.first || kk > 0) ? 1u : 0u);
                }
                __syncwarp();
                commit(kPVDone + h);
                if (now.closes)
                    commit(kVEmpty + stage);
                const Step after = next.valid ? it.next(pieces, count) : next;
                // S(j + 2) overwrites P(j); the wait is also this block's last
                if (!wait(kPVDone + h, phase))
                    break;
                if (after.valid && !scores(j + 2, after))
                    break;
                now = next;
                next = after;
            }
        }
    } else if (kCodes && warp >= 12) {
        setmaxnreg_dec<(kCodes ? Lay::kRegsConvert : 24)>();
        // ===================== codes into f16: keys 32 w .. of every tile ===============
        if constexpr (kCodes) {
            const int key0 = (warp - 12) * kRunKeys;
            const int2* info = reinterpret_cast<const int2*>(smem + Lay::kSlotInfo);
            for (int u = 0;; ++u) {
                const int slot = u % kRing;
                if (!mbar_wait_warp(&bar[kCodeFull + slot], (u / kRing) & 1, misc, a.err))
                    break;
                const int2 what = info[slot];
                if (what.x < 0)
                    break;
                const int v = what.x & 1, tile = what.x >> 1;
                const int st = v ? 0 : tile & 1;
                const uint32_t turn = v ? tile : tile >> 1;
                const bool ok = mbar_wait_warp(&bar[(v ? kVEmpty : kKEmpty) + st], (turn & 1) ^ 1u, misc, a.err);
                if (ok) {
                    uint8_t* mat = smem + (v ? Lay::kV : Lay::kK) + st * Lay::kMat;
                    const uint8_t* from = smem + Lay::kCodeRing + slot * Lay::kCodeTile + key0 * Lay::kRowBytes;
                    if (what.y >= key0 + kRunKeys)
                        convert_run<KIND, false>(mat, Lay::kBlock, from, key0, kRunKeys, lane);
                    else
                        convert_run<KIND, true>(mat, Lay::kBlock, from, key0, what.y - key0, lane);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (ok)
                        mbar_arrive(&bar[(v ? kVFull : kKFull) + st]);
                    mbar_arrive(&bar[kCodeEmpty + slot]);
                }
            }
        }
    } else {
        const int half = (warp - 4) >> 2;
        const int w4 = warp & 3;
        const int r = w4 * 32 + lane;
        const uint32_t trow = tmem + (uint32_t(w4 * 32) << 16);
        const uint32_t ts = trow + col_s(half), to = trow + col_o(half);
        const float c2l = a.scale_log2;
        uint8_t* mat = smem + Lay::kQ + half * Lay::kMat;
        // ===================== softmax: one warpgroup per half =====================
        setmaxnreg_inc<Lay::kRegsSoftmax>();
        // (What a piece needs again at its end is read again from shared memory: the fold
        // needs every register it has.)
        int j0 = 0, g0 = 0;                              // the block's steps and tiles before this piece
        for (int i = 0, tiles, steps; i < count; ++i, j0 += steps, g0 += tiles) {
            const volatile Piece& pc = pieces[i];
            const int n = pc.len, tile0 = pc.k0;
            const bool pair = pc.rows > 128;
            tiles = pc.k1 - tile0;
            steps = pair ? 2 * tiles : tiles;
            // region 0: the half that takes the piece's first step
            const int region = half ^ (j0 & 1);
            const int mine = (steps - region + 1) >> 1;
            // this thread's row
            const int f = pair ? pc.rb * 256 + region * 128 + r : r;
            const bool live = f < pc.rows;
            // (Rows behind the last take another's query: they see nothing, and a branch around
            // the loads would have each wait for the one before, 6 us.)
            const int fr = live ? f : 0;
            const int in = a.by_R.of(fr), x = fr - in * a.R, b = pc.first + in;
            const int64_t q_at = ((int64_t(b) * a.H_q + pc.h * a.G) * a.L + x) * D;
            const int ctx = __ldg(a.context_lens + b);
            if (mine == 0) {
                if (live)
                    __stcg(a.state_ml + (int64_t(pc.item) + c) * 256 + region * 128 + r, make_float2(-INFINITY, 0.f));
                continue;
            }
            // ---- the rows of Q, 16 bytes a lane, swizzled as TMA would
            {
                constexpr int kChunks = D / 8;           // 16-byte chunks of a row
                constexpr int kPer = 32 / kChunks;       // rows a round
                constexpr int kRounds = 32 / kPer;
                const int ch = lane % kChunks;
                auto place = [&](int i) {                // of round i's
                    const int rr = w4 * 32 + i * kPer + lane / kChunks;
                    return reinterpret_cast<uint4*>(mat + (ch >> 3) * Lay::kBlock + rr * 128 +
                                                    (((ch & 7) ^ (rr & 7)) << 4));
                };
#pragma unroll 2
                for (int i = 0; i < kRounds; ++i) {
                    const int64_t at = __shfl_sync(0xffffffffu, q_at, i * kPer + lane / kChunks);
                    cp_async_16(place(i), a.q + at + ch * 8, 16);
                }
                cp_async_commit();
                cp_async_wait_group<0>();
                if constexpr (kCodes) {                  // each lane what it has copied
#pragma unroll 2
                    for (int i = 0; i < kRounds; ++i) {
                        uint4 v = *place(i);
                        v = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z),
                                       bf16x2_to_f16x2(v.w));
                        *place(i) = KIND == kQ4Pool ? apart(v) : v;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[kQFull + half]);
            }
            const int cap = a.max_pages * a.block_ps;
            int lim = (ctx < 0 ? 0 : ctx > cap ? cap : ctx) - a.L + x - a.by_L.of(x) * a.L;
            lim = live ? min(n - 1, lim) : -1;
            float m_used = -INFINITY, l = 0.f;
            for (int u = 0; u < mine; ++u) {
                const int j = j0 + 2 * u + region;       // step of the block: j & 1 == half
                const int in_piece = 2 * u + region;
                const int tile = pair ? u : in_piece;    // of the piece
                const int g = g0 + tile;
                const bool opens = !pair || region == 0;
                const uint32_t phase = (j >> 1) & 1;
                mbar_wait_warp(&bar[kSFull + half], phase, misc, a.err);
                tc_fence_after();
                const int key0 = (tile0 + tile) * kKeys;
                uint32_t sv[128];
                float* sc = reinterpret_cast<float*>(sv);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    tmem_ld32(ts + 32u * w, sv + 32 * w);
                tmem_wait_ld();
                if (key0 + kKeys - 1 > lim) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int nv = lim - (key0 + 32 * w) + 1;
                        const uint32_t vis = nv >= 32 ? 0xffffffffu : nv <= 0 ? 0u : (1u << nv) - 1u;
#pragma unroll
                        for (int kq = 0; kq < 32; ++kq)
                            sc[32 * w + kq] = (vis >> kq) & 1u ? sc[32 * w + kq] : -INFINITY;
                    }
                }
                float m8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m8[i] = -INFINITY;
#pragma unroll
                for (int kq = 0; kq < 128; kq += 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        m8[i] = fmaxf(m8[i], sc[kq + i]);
                const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                       fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                const float mxs = mx * c2l;
                const bool need = mxs > m_used + kRescaleLog2 || (m_used == -INFINITY && mxs > -INFINITY);
                float factor = 1.f;
                if (need) {
                    factor = m_used == -INFINITY ? 0.f : fast_exp2(m_used - mxs);
                    m_used = mxs;
                    l *= factor;
                }
                const float mu = m_used == -INFINITY ? 0.f : m_used;
                const float2 cc = make_float2(c2l, c2l), nmu2 = make_float2(-mu, -mu);
                float2 lsum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                  make_float2(0.f, 0.f)};
                auto exp_store = [&](int hf) {
                    uint32_t pk[32];
#pragma unroll
                    for (int kq = 0; kq < 32; ++kq) {
                        const float2 v =
                            __ffma2_rn(make_float2(sc[64 * hf + 2 * kq], sc[64 * hf + 2 * kq + 1]), cc, nmu2);
                        const float2 pp = make_float2(fast_exp2(v.x), fast_exp2(v.y));
                        lsum[kq & 3] = __fadd2_rn(lsum[kq & 3], pp);
                        pk[kq] = kCodes ? pack_f16x2(pp.x, pp.y) : pack_bf16x2(pp.x, pp.y);
                    }
                    tmem_st32(ts + kPCol + 32u * hf, pk);
                };
                exp_store(1);
                exp_store(0);
                {
                    const float2 t2 = __fadd2_rn(__fadd2_rn(lsum[0], lsum[1]), __fadd2_rn(lsum[2], lsum[3]));
                    l += t2.x + t2.y;
                }
                // O holds the half's earlier tiles of the piece; the product of the last
                // of them has ended before S of this one began
                if (u > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        uint32_t ov[32];
                        tmem_ld32(to + 32u * q4, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int kq = 0; kq < 32; ++kq)
                            ov[kq] = __float_as_uint(__uint_as_float(ov[kq]) * factor);
                        tmem_st32(to + 32u * q4, ov);
                    }
                }
                tmem_wait_st();
                // V rows past the prefix hold whatever the page or the stage held: zeros
                // before either half's product with them (codes: written as zeros)
                if (!kCodes && opens && n < key0 + kKeys) {
                    mbar_wait_bounded(&bar[kVFull + (g & 1)], (g >> 1) & 1, misc, a.err);
                    const int z = n - key0;
                    uint8_t* vb = smem + Lay::kV + (g & 1) * Lay::kMat;
#pragma unroll 1
                    for (int idx = r; idx < (kKeys - z) * (D / 8); idx += 128) {
                        const int zr = z + idx / (D / 8), ch = idx % (D / 8);
                        *reinterpret_cast<uint4*>(vb + (ch >> 3) * Lay::kBlock + zr * 128 +
                                                  (((ch & 7) ^ (zr & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[kPFull + half]);
            }
            // ---- the state: through this warp's own rows of Q (their last product has
            // ended), so that whole 128-byte pieces of rows leave together
            mbar_wait_warp(&bar[kPVDone + half], ((j0 + 2 * (mine - 1) + region) >> 1) & 1, misc, a.err);
            tc_fence_after();
            const bool good = misc[0] == 0;
            const int64_t place = (int64_t(pc.item) + c) * 256 + region * 128;
            if (live && good)
                __stcg(a.state_ml + place + r, make_float2(m_used, l));
            uint8_t* stage = mat + w4 * 32 * 128;
            float* rows_out = a.state + (place + w4 * 32) * D;
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) {
                uint32_t ov[32];
                tmem_ld32(to + 32u * q4, ov);
                tmem_wait_ld();
#pragma unroll
                for (int cq = 0; cq < 8; ++cq) {
                    // elements 4 cq .. 4 cq + 3; 4-bit rows: places 2 i or 2 i + 1 of the 8
                    constexpr bool kApart = KIND == kQ4Pool;
                    const int at = kApart ? 8 * (cq >> 1) + (cq & 1) : 4 * cq, by = kApart ? 2 : 1;
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((cq ^ (lane & 7)) << 4)) =
                        make_uint4(ov[at], ov[at + by], ov[at + 2 * by], ov[at + 3 * by]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = i * 4 + (lane >> 3), cq = lane & 7;
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + ((cq ^ (row & 7)) << 4));
                    const bool there = __shfl_sync(0xffffffffu, int(live), row) != 0;
                    if (there && good)
                        __stcg(reinterpret_cast<uint4*>(rows_out + row * D + q4 * 32 + cq * 4), v);
                }
                __syncwarp();
            }
            tc_fence_before();
        }
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// (Where code runs once a block, its size counts: loops are kept rolled below. Unrolled by
// the compiler they cost 0.3 to 2 us a call.)

// The last step joins the states that the prefix's pieces and the segment behind it left
// for a row: by a.share warps of a block (a power of two), each some of the pieces. Where
// they lie is read from what the two kernels before noted down, row by row: found again
// from the call's tables, by every warp, it took 2 to 6 us (few of these blocks fit beside
// the few-row kernel's, so it was not hidden before the wait). A chain of two reads: the
// notes, then the states' (m, l) together with the first states.
// kMergeWarpsPerSM bounds the warps a row gets. 32 bf16 requests behind 16384 keys, 64
// e4m3 requests (us, whole calls), 40 warps: 34.0, 63.9; 24: 34.4, 67.7; 48: 35.8, 65.2;
// 64 warps of fewer registers 43.9, 76.2.
constexpr int kMergeWarps = 8, kMergeThreads = 32 * kMergeWarps, kMergeWarpsPerSM = 40;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) prefix_merge_kernel(const PrefixMergeArgs a)
{
    __shared__ float4 sums[kMergeWarps][32];
    __shared__ float2 row_ml[kMergeWarps];               // (max, sum) of each warp's pieces
    const PrefixKernelArgs& k = a.prefix_args;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = a.share, sub = warp & (share - 1);
    const int row = (int(blockIdx.x) * kMergeWarps + warp) / share;   // of [B, H_kv, R]
    const bool live = row < k.B * k.H_kv * k.R;
    const int bh = live ? k.by_R.of(row) : 0, x = live ? row - bh * k.R : 0;
    const int b = k.by_H.of(bh), h = bh - b * k.H_kv;
    int np = 0, ns = 0, twice = 0;                       // states of the prefix, of the segment
    int64_t p_row = 0;                                   // the row's in the prefix's first state
    const int slot = suffix_slot_floats(D, a.row_tiles);
    const int xr = x % kSegmentRows;
    const int seg = bh * a.MS + x / kSegmentRows;
    const float* s_at = a.suffix_state;
    grid_dependency_wait();
    grid_launch_dependents();
    if (live) {
        const int4 note = __ldcg(k.note_row + row);
        const int2 blocks = __ldcg(a.note_segment + seg);
        np = note.y;
        twice = note.w;                                  // both halves hold the rows
        p_row = int64_t(note.x) * 256 + note.z;
        ns = blocks.y - blocks.x + 1;
        s_at += (int64_t(seg) + blocks.x) * slot;
    }
    const int pieces = np + ns;
    auto p_place = [&](int t) { return p_row + int64_t(t >> twice) * 256 + ((t & twice) << 7); };

    // ---- this warp's pieces sub, sub + share, ...: 32 at a time, their (m, l) a lane
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 4;                           // states on their way
    auto fetch = [&](int t, float4* v) {                 // of pieces t, t + share, ...
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i, t += share) {
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < pieces) {
                const float* at = t < np ? k.state + p_place(t) * D : s_at + int64_t(t - np) * slot + xr * D;
                if constexpr (D == 128) {
                    v[i] = __ldcg(reinterpret_cast<const float4*>(at) + lane);
                } else {
                    const float2 x2 = __ldcg(reinterpret_cast<const float2*>(at) + lane);
                    v[i].x = x2.x;
                    v[i].y = x2.y;
                }
            }
        }
    };
#pragma unroll 1
    for (int t0 = sub; t0 < pieces; t0 += 32 * share) {
        const int mine = t0 + lane * share;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine < pieces)
            ml = __ldcg(mine < np ? k.state_ml + p_place(mine)
                                  : reinterpret_cast<const float2*>(s_at + int64_t(mine - np) * slot +
                                                                    8 * a.row_tiles * D) + xr);
        float4 v[kAtOnce];
        fetch(t0, v);
        float m = fmaxf(top, ml.x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        // nothing seen: the state was not written, and counts for nothing (scores that are
        // all NaN have no largest either: their sum is NaN, and makes this one NaN)
        const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m);
        const float old = top == -INFINITY ? 0.f : fast_exp2(top - m);
        float add = w * ml.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            add += __shfl_xor_sync(0xffffffffu, add, off);
        sum = sum * old + add;
        o.x *= old;
        o.y *= old;
        o.z *= old;
        o.w *= old;
        top = m;
        const int n = min(32, (pieces - t0 + share - 1) / share);
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kAtOnce) {
            if (i0 > 0)
                fetch(t0 + i0 * share, v);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i0 + i);     // 0 behind the last
                if (wi != 0.f) {                         // (NaN too; what was not written is not used)
                    o.x = fmaf(wi, v[i].x, o.x);
                    o.y = fmaf(wi, v[i].y, o.y);
                    o.z = fmaf(wi, v[i].z, o.z);
                    o.w = fmaf(wi, v[i].w, o.w);
                }
            }
        }
    }
    if (share > 1) {
        sums[warp][lane] = o;
        if (lane == 0)
            row_ml[warp] = make_float2(top, sum);
        __syncthreads();
        if (sub != 0)
            return;
        float m = top;
#pragma unroll 1
        for (int w = 1; w < share; ++w)
            m = fmaxf(m, row_ml[warp + w].x);
        const float f = top == -INFINITY ? 0.f : fast_exp2(top - m);
        sum *= f;
        o.x *= f;
        o.y *= f;
        o.z *= f;
        o.w *= f;
#pragma unroll 1
        for (int w = 1; w < share; ++w) {
            const float2 ml = row_ml[warp + w];
            const float fw = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m);
            const float4 v = sums[warp + w][lane];
            sum = fmaf(fw, ml.y, sum);
            o.x = fmaf(fw, v.x, o.x);
            o.y = fmaf(fw, v.y, o.y);
            o.z = fmaf(fw, v.z, o.z);
            o.w = fmaf(fw, v.w, o.w);
        }
    }
    if (live) {
        const float inv = sum == 0.f ? 0.f : a.out_scale / sum;     // NaN stays
        uint16_t* dst = a.out + ((int64_t(b) * k.H_q + h * k.G) * k.L + x) * D;
        if constexpr (D == 128)
            reinterpret_cast<uint2*>(dst)[lane] =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        else
            reinterpret_cast<uint32_t*>(dst)[lane] = pack_bf16x2(o.x * inv, o.y * inv);
    }
}

}  // namespace

size_t prefix_smem_bytes(int D, int kind, int count)
{
    const int fixed = kind == kE4m3Pool ? Layout<128, kE4m3Pool>::kGroups
                      : kind == kQ4Pool ? Layout<128, kQ4Pool>::kGroups
                      : D == 64         ? Layout<64, kBf16Pool>::kGroups
                                        : Layout<128, kBf16Pool>::kGroups;
    return size_t(fixed) + size_t(count) * sizeof(Group) + 1024;
}

size_t prefix_state_bytes(const pa_shape& s, int64_t items, int grid, size_t* ml_off, size_t* pieces_off)
{
    const size_t slots = size_t(items + grid);
    *ml_off = slots * 256 * size_t(s.head_dim) * sizeof(float);
    *pieces_off = *ml_off + slots * 256 * sizeof(float2);
    return *pieces_off + (items > kMaxPieces ? size_t(items) * size_t(grid) * sizeof(Piece) : 0);
}

namespace {

using PrefixKernel = void (*)(CUtensorMap, CUtensorMap, PrefixKernelArgs);

int prefix_instance(int D, int kind) { return kind == kE4m3Pool ? 2 : kind == kQ4Pool ? 3 : D == 64 ? 0 : 1; }

PrefixKernel prefix_kernel_of(int which)
{
    static const PrefixKernel kernels[4] = {prefix_kernel<64, kBf16Pool>, prefix_kernel<128, kBf16Pool>,
                                            prefix_kernel<128, kE4m3Pool>, prefix_kernel<128, kQ4Pool>};
    return kernels[which];
}

int prefix_threads(int kind)
{
    return kind == kBf16Pool ? Layout<128, kBf16Pool>::kThreads : Layout<128, kE4m3Pool>::kThreads;
}

}  // namespace

cudaError_t prepare_prefix(int D, int kind, int device)
{
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev][4];
    static std::atomic<int> regs_ok[kMaxDev][4];
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    const int which = prefix_instance(D, kind), threads = prefix_threads(kind);
    const void* fn = reinterpret_cast<const void*>(prefix_kernel_of(which));
    const int first = kind == kBf16Pool ? Layout<128, kBf16Pool>::kRegsFirst : Layout<128, kE4m3Pool>::kRegsFirst;
    const int most = kind == kBf16Pool ? Layout<128, kBf16Pool>::kRegsSoftmax : Layout<128, kE4m3Pool>::kRegsSoftmax;
    const int sum = kind == kBf16Pool ? Layout<128, kBf16Pool>::kRegsSum : Layout<128, kE4m3Pool>::kRegsSum;
    // setmaxnreg draws on the registers that the block was launched with
    int rk = regs_ok[device][which].load(std::memory_order_relaxed);
    if (rk == 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, fn);
        if (e != cudaSuccess)
            return e;
        rk = fa.numRegs >= first && fa.numRegs <= most && sum <= threads * fa.numRegs ? 1 : 2;
        regs_ok[device][which].store(rk, std::memory_order_relaxed);
    }
    if (rk != 1)
        return cudaErrorNotSupported;
    return raise_smem_limit(fn, &raised[device][which]);
}

cudaError_t launch_prefix(const CUtensorMap& key_map, const CUtensorMap& value_map, const PrefixKernelArgs& a,
                          int D, int kind, int grid, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(prefix_threads(kind));
    cfg.dynamicSmemBytes = prefix_smem_bytes(D, kind, a.prefix.count);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_kernel_of(prefix_instance(D, kind)), key_map, value_map, a);
}

cudaError_t launch_prefix_merge(PrefixMergeArgs a, int D, int sm_count, cudaStream_t stream)
{
    const PrefixKernelArgs& k = a.prefix_args;
    const int64_t rows = int64_t(k.B) * k.H_kv * k.R;
    a.share = kMergeWarps;
    while (a.share > 1 && rows * a.share > int64_t(sm_count) * kMergeWarpsPerSM)
        a.share /= 2;
    const int64_t blocks = (rows * a.share + kMergeWarps - 1) / kMergeWarps;
    if (blocks <= 0 || blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, D == 64 ? prefix_merge_kernel<64> : prefix_merge_kernel<128>, a);
}

}  // namespace pa
