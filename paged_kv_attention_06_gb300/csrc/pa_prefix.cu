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
//   * warp 0: K tiles, warp 2: V tiles by TMA, page by page, two stages each;
//   * warp 1 (one elected thread): the tcgen05.mma chain;
//   * warps 4-7 and 8-11: the query rows of a piece into shared memory, the softmax
//     (P over the upper half of the scores' columns in TMEM, rounded to bf16: its error,
//     2^-9 of a term, averages out below the output's own rounding), the states.
// TMEM (512 columns): S_0, S_1, O_0, O_1 (128 each).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefix.cuh"
#include "pa_split.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kKeys = 128;            // keys per tile
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;
constexpr int kRegsProducer = 128;
constexpr int kRegsSoftmax = 184;
static_assert(128 * kRegsProducer + 256 * kRegsSoftmax <= 65536, "register split");

__host__ __device__ constexpr uint32_t col_s(int half) { return uint32_t(half * 128); }
__host__ __device__ constexpr uint32_t col_o(int half) { return uint32_t(256 + half * 128); }
constexpr uint32_t kPCol = 64;

template <int D>
struct Layout {
    static constexpr int kBlock = 128 * 128;            // 128 rows x 64 bf16 (128 B)
    static constexpr int kMat = D / 64 * kBlock;        // 128 x D bf16, [column block][row][128 B]
    static constexpr int kQ = 0;                        // [half]
    static constexpr int kK = kQ + 2 * kMat;            // 2 stages
    static constexpr int kV = kK + 2 * kMat;            // 2 stages
    static constexpr int kBar = kV + 2 * kMat;
    static constexpr int kNumBars = 16;
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kMisc = kTmemSlot + 16;
    static constexpr int kGroups = kMisc + 16;          // Group[count]
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
static_assert(kPVDone + 1 < Layout<128>::kNumBars, "barrier count");

// A tile weighs kTileUnits, an item kItemUnits more (its rows, its state: about two
// tiles' time); a tile belongs to the block whose range holds its first unit. A block has
// at least kLeastUnits (but the last), so that no range lies inside a tile.
constexpr int kTileUnits = 4;
constexpr int kItemUnits = 8;
constexpr int kLeastUnits = 8;

// One prefix: where its units and items start, its keys, its rows for one KV head.
struct Group {
    long long us;
    int item, items, len, first, rows, tiles;
    __device__ __forceinline__ long long item_units() const { return (long long)tiles * kTileUnits + kItemUnits; }
};

// *bad: the starts do not ascend within the batch.
__device__ __forceinline__ Group group_at(const PrefixKernelArgs& a, int p, bool* bad)
{
    Group g;
    g.first = __ldg(a.prefix.starts + p);
    const int end = __ldg(a.prefix.starts + p + 1);
    *bad = g.first < 0 || end < g.first || end > a.B;
    g.len = prefix_len(a.prefix, p);
    g.tiles = (g.len + kKeys - 1) / kKeys;
    g.rows = *bad ? 0 : (end - g.first) * a.R;
    g.items = g.tiles > 0 ? a.H_kv * ((g.rows + 255) / 256) : 0;
    g.us = 0;
    g.item = 0;
    return g;
}

// Blocks that take part, of U units.
__device__ __forceinline__ long long working_blocks(long long U, int grid)
{
    const long long most = U / kLeastUnits;
    return most < 1 ? 1 : most < grid ? most : grid;
}
__device__ __forceinline__ long long range_start(long long c, long long U, long long G) { return c * U / G; }
__device__ __forceinline__ int block_of(long long x, long long U, long long G) { return int(((x + 1) * G - 1) / U); }

// The part of an item in a block's range of units.
struct Piece {
    int p, item, h, rb;      // prefix, item of all, KV head, block of 256 rows
    int k0, k1;              // tiles
};
struct Cursor {
    int p, i;                // the next item: the i-th of prefix p
    __device__ __forceinline__ bool next(const Group* groups, int count, long long s, long long e, Piece& out)
    {
        for (;;) {
            if (p >= count)
                return false;
            const Group& g = groups[p];
            if (i >= g.items) {
                ++p;
                i = 0;
                continue;
            }
            const long long us = g.us + i * g.item_units();
            if (us >= e)
                return false;
            auto first_at = [&](long long x) {
                const long long d = x - us - kItemUnits;
                const long long k = d <= 0 ? 0 : (d + kTileUnits - 1) / kTileUnits;
                return int(k > g.tiles ? g.tiles : k);
            };
            out.k0 = first_at(s);
            out.k1 = first_at(e);
            const int blocks = (g.rows + 255) / 256;
            out.p = p;
            out.item = g.item + i;
            out.h = i / blocks;
            out.rb = i - out.h * blocks;
            ++i;
            if (out.k0 < out.k1)
                return true;
        }
    }
};

// The products' steps, in order: a step is one warpgroup's (half's) work on one tile.
// Half j & 1 takes step j; `first` / `last` of its piece for that half, `opens` /
// `closes` the tile's loads.
struct Step {
    int g;                   // tile of the block's stream
    bool first, opens, closes, valid;
};
struct StepIter {
    Cursor cur;
    Piece piece;
    int k, g, sub, done;     // next tile of the piece, of the stream; steps of the tile; of the piece
    bool have, pair;
    __device__ __forceinline__ Step next(const Group* groups, int count, long long s, long long e)
    {
        Step st;
        st.valid = false;
        if (!have || k >= piece.k1) {
            if (!cur.next(groups, count, s, e, piece))
                return st;
            have = true;
            k = piece.k0;
            sub = done = 0;
            pair = groups[piece.p].rows > 128;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap value_map,
                  const PrefixKernelArgs a)
{
    using Lay = Layout<D>;
    constexpr int kBlocks = D / 64;                      // 128-byte column blocks of a row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kTmemSlot);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + Lay::kMisc);
    Group* groups = reinterpret_cast<Group*>(smem + Lay::kGroups);
    __shared__ long long total_units;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int count = a.prefix.count;

    grid_dependency_wait();
    grid_launch_dependents();
    // ---- the prefixes' places in the stream ---------------------------------------
    if (warp == 0) {
        long long us = 0;
        int item = 0;
        bool bad = false;
        for (int base = 0; base < count; base += 32) {
            const int p = base + lane;
            Group g;
            g.items = 0;
            g.tiles = 0;
            if (p < count) {
                bool no;
                g = group_at(a, p, &no);
                bad |= no;
                const int n = __ldg(a.prefix.lens + p);
                if (blockIdx.x == 0 && (n < 0 || n > a.prefix.cap))
                    atomicOr(a.err, PA_DEVERR_CONTEXT_LEN_BIT);
            }
            const long long units = g.items * g.item_units();
            long long incl_u = units;
            int incl_i = g.items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, incl_u, o);
                const int v = __shfl_up_sync(0xffffffffu, incl_i, o);
                if (lane >= o) {
                    incl_u += u;
                    incl_i += v;
                }
            }
            if (p < count) {
                g.us = us + incl_u - units;
                g.item = item + incl_i - g.items;
                groups[p] = g;
            }
            us += __shfl_sync(0xffffffffu, incl_u, 31);
            item += __shfl_sync(0xffffffffu, incl_i, 31);
        }
        // Rows counted twice would have more states than there is room for: none then.
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            total_units = bad ? 0 : us;
            if (bad && blockIdx.x == 0)
                atomicOr(a.err, PA_DEVERR_PREFIX_BIT);
        }
    }
    __syncthreads();
    const long long U = total_units;
    const long long G = working_blocks(U, int(gridDim.x));
    const int c = int(blockIdx.x);
    if (U == 0 || c >= G)
        return;
    const long long s = range_start(c, U, G), e = range_start(c + 1, U, G);
    Cursor start;
    {
        int lo = 0, hi = count;                          // the last prefix that starts at or before s
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (groups[mid].us <= s)
                lo = mid;
            else
                hi = mid;
        }
        start.p = lo;
        start.i = groups[lo].items > 0 ? int((s - groups[lo].us) / groups[lo].item_units()) : 0;
    }

    const uint32_t sQ = smem_u32(smem + Lay::kQ), sK = smem_u32(smem + Lay::kK), sV = smem_u32(smem + Lay::kV);
    if (threadIdx.x == 0) {
        misc[0] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[kQFull + i], 4);              // one arrival per warp
            mbar_init(&bar[kKFull + i], 1);
            mbar_init(&bar[kKEmpty + i], 1);
            mbar_init(&bar[kVFull + i], 1);
            mbar_init(&bar[kVEmpty + i], 1);
            mbar_init(&bar[kSFull + i], 1);
            mbar_init(&bar[kPFull + i], 4);
            mbar_init(&bar[kPVDone + i], 1);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        setmaxnreg_dec<kRegsProducer>();
        if (warp == 0 || warp == 2) {
            // ===================== K (warp 0) and V (warp 2) tiles ===================
            const bool is_v = warp == 2;
            const CUtensorMap* map = is_v ? &value_map : &key_map;
            uint8_t* to = smem + (is_v ? Lay::kV : Lay::kK);
            const int full = is_v ? kVFull : kKFull, empty = is_v ? kVEmpty : kKEmpty;
            const uint64_t policy = l2_policy_evict_last();  // the item's other row blocks read it too
            if (lane == 0)
                prefetch_tensormap(map);
            const int box = a.box_rows;                  // min(page size, 128), at least 8
            Cursor cur = start;
            Piece pc;
            int g = 0;
            while (cur.next(groups, count, s, e, pc)) {
                const int n = groups[pc.p].len;
                for (int k = pc.k0; k < pc.k1; ++k, ++g) {
                    const int key0 = k * kKeys;
                    const int boxes = (min(n, key0 + kKeys) - key0 + box - 1) / box;
                    const int tok = key0 + lane * box;
                    int phys = lane < boxes ? __ldg(a.prefix.table + int64_t(pc.p) * a.prefix.pages + tok / a.ps) : 0;
                    const int st = g & 1;
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
                            const int row = (phys * a.H_kv + pc.h) * a.ps + tok % a.ps;
                            uint8_t* dst = to + st * Lay::kMat + lane * box * 128;
#pragma unroll
                            for (int x = 0; x < kBlocks; ++x)
                                tma_load_2d(dst + x * Lay::kBlock, map, 64 * x, row, &bar[full + st], policy);
                        }
                    }
                    __syncwarp();
                }
            }
            // No copy may still be landing when the block exits.
            for (int i = max(0, g - 2); i < g; ++i)
                mbar_wait_bounded(&bar[full + (i & 1)], (i >> 1) & 1, misc, a.err);
        } else if (warp == 1) {
            // ===================== MMA issue (one elected thread) =====================
            const bool leader = elect_one();
            const uint32_t idesc_s = idesc_bf16_f32(128, kKeys, 0);
            const uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
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
            int pieces[2] = {0, 0};                      // query tiles waited for, by half
            auto scores = [&](int j, const Step& st) {
                const int h = j & 1, stage = st.g & 1;
                if (st.first) {
                    if (!wait(kQFull + h, pieces[h] & 1))
                        return false;
                    ++pieces[h];
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
            it.cur = start;
            it.have = false;
            it.g = 0;
            Step now = it.next(groups, count, s, e), next = it.next(groups, count, s, e);
            bool ok = now.valid && scores(0, now) && (!next.valid || scores(1, next));
            int j = 0;
            for (; ok && now.valid; ++j) {
                const int h = j & 1, stage = now.g & 1;
                const uint32_t phase = (j >> 1) & 1;
                if (!wait(kPFull + h, phase) || !wait(kVFull + stage, (now.g >> 1) & 1))
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
                const Step after = next.valid ? it.next(groups, count, s, e) : next;
                // S(j + 2) overwrites P(j); the wait is also this block's last
                if (!wait(kPVDone + h, phase))
                    break;
                if (after.valid && !scores(j + 2, after))
                    break;
                now = next;
                next = after;
            }
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ===================== softmax: one warpgroup per half =====================
        const int half = (warp - 4) >> 2;
        const int w4 = warp & 3;
        const int r = w4 * 32 + lane;
        const uint32_t trow = tmem + (uint32_t(w4 * 32) << 16);
        const uint32_t ts = trow + col_s(half), to = trow + col_o(half);
        const float c2l = a.scale_log2;
        uint8_t* mat = smem + Lay::kQ + half * Lay::kMat;
        Cursor cur = start;
        Piece pc;
        int j0 = 0;                                      // the block's steps before this piece
        int g0 = 0;                                      // and tiles
        while (cur.next(groups, count, s, e, pc)) {
            const Group& gr = groups[pc.p];
            const int n = gr.len;
            const bool pair = gr.rows > 128;
            const int tiles = pc.k1 - pc.k0;
            const int steps = pair ? 2 * tiles : tiles;
            // region 0: the half that takes the piece's first step
            const int region = half ^ (j0 & 1);
            const int mine = (steps - region + 1) >> 1;
            // this thread's row
            const int f = pair ? pc.rb * 256 + region * 128 + r : r;
            const bool live = f < gr.rows;
            const int b = live ? gr.first + f / a.R : 0, x = live ? f % a.R : 0;
            int lim = -1;                                // its last visible key
            int64_t q_at = 0;
            if (live) {
                const int cap = a.max_pages * a.block_ps;
                int ctx = __ldg(a.context_lens + b);
                ctx = ctx < 0 ? 0 : ctx > cap ? cap : ctx;
                lim = min(n, ctx - a.L + x % a.L + 1) - 1;
                q_at = ((int64_t(b) * a.H_q + pc.h * a.G) * a.L + x) * D;
            }
            const int64_t slot = int64_t(pc.item) + c;
            float2* ml = a.state_ml + slot * 256 + region * 128;
            if (mine == 0) {
                if (live)
                    __stcg(ml + r, make_float2(-INFINITY, 0.f));
                j0 += steps;
                g0 += tiles;
                continue;
            }
            // ---- the rows of Q, 16 bytes a lane, swizzled as TMA would
            {
                constexpr int kChunks = D / 8;           // 16-byte chunks of a row
                constexpr int kPer = 32 / kChunks;       // rows a round
#pragma unroll
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int row = i * kPer + lane / kChunks, ch = lane % kChunks;
                    const int64_t at = __shfl_sync(0xffffffffu, q_at, row);
                    const bool there = __shfl_sync(0xffffffffu, int(live), row) != 0;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (there)
                        v = *reinterpret_cast<const uint4*>(a.q + at + ch * 8);
                    const int rr = w4 * 32 + row;
                    *reinterpret_cast<uint4*>(mat + (ch >> 3) * Lay::kBlock + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[kQFull + half]);
            }
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
                const int key0 = (pc.k0 + tile) * kKeys;
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
                        pk[kq] = pack_bf16x2(pp.x, pp.y);
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
                // before either half's product with them
                if (opens && n < key0 + kKeys) {
                    mbar_wait_bounded(&bar[kVFull + (g & 1)], (g >> 1) & 1, misc, a.err);
                    const int z = n - key0;
                    uint8_t* vb = smem + Lay::kV + (g & 1) * Lay::kMat;
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
            if (live && good)
                __stcg(ml + r, make_float2(m_used, l));
            uint8_t* stage = mat + w4 * 32 * 128;
            float* rows_out = a.state + (slot * 256 + region * 128 + w4 * 32) * D;
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) {
                uint32_t ov[32];
                tmem_ld32(to + 32u * q4, ov);
                tmem_wait_ld();
#pragma unroll
                for (int cq = 0; cq < 8; ++cq)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((cq ^ (lane & 7)) << 4)) =
                        make_uint4(ov[4 * cq], ov[4 * cq + 1], ov[4 * cq + 2], ov[4 * cq + 3]);
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
            j0 += steps;
            g0 += tiles;
        }
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The last step: one block per query row joins the states that the prefix's pieces and
// the row's own segment left. Everything before the wait is from the call's inputs, so
// it runs while the kernels before are at work.
constexpr int kMergeThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const PrefixMergeArgs a)
{
    extern __shared__ float weights[];                   // [pieces]
    __shared__ float4 sums[kMergeThreads / 32][32];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ long long red_units[2][kMergeThreads / 32];
    __shared__ int red_items[kMergeThreads / 32];
    grid_launch_dependents();
    const PrefixKernelArgs& k = a.prefix_args;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;                      // of [B, H_kv, R]
    const int bh = int(row / k.R), x = int(row - int64_t(bh) * k.R);
    const int b = bh / k.H_kv, h = bh - b * k.H_kv;

    // ---- the prefix's pieces
    long long U = 0, us = 0;
    int item = 0;
    bool bad = false;
    for (int p = threadIdx.x; p < k.prefix.count; p += kMergeThreads) {
        bool no;
        const Group g = group_at(k, p, &no);
        bad |= no;
        const long long units = g.items * g.item_units();
        // the prefixes before b's end at or before it
        const bool before = g.items > 0 && g.first + g.rows / k.R <= b;
        U += units;
        us += before ? units : 0;
        item += before ? g.items : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        U += __shfl_xor_sync(0xffffffffu, U, o);
        us += __shfl_xor_sync(0xffffffffu, us, o);
        item += __shfl_xor_sync(0xffffffffu, item, o);
    }
    if (lane == 0) {
        red_units[0][warp] = U;
        red_units[1][warp] = us;
        red_items[warp] = item;
    }
    // ---- the segment's pieces behind it
    const int cap = k.max_pages * k.block_ps;
    auto granules = [&](int q) {
        int n = __ldcg(k.context_lens + q);
        n = n < 0 ? 0 : n > cap ? cap : n;
        return suffix_granules(n, min(prefix_len_of(k.prefix, q), n), a.box_rows, a.tile_keys);
    };
    int total = 0, ahead = 0;
    for (int q = threadIdx.x; q < k.B; q += kMergeThreads) {
        const int gs = granules(q) * a.per_req;
        total += gs;
        ahead += q < b ? gs : 0;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    ahead = __reduce_add_sync(0xffffffffu, ahead);
    __shared__ int red_gran[2][kMergeThreads / 32];
    if (lane == 0) {
        red_gran[0][warp] = total;
        red_gran[1][warp] = ahead;
    }
    bad = __syncthreads_or(bad);
    U = us = 0;
    item = total = ahead = 0;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) {
        U += red_units[0][w];
        us += red_units[1][w];
        item += red_items[w];
        total += red_gran[0][w];
        ahead += red_gran[1][w];
    }
    int np = 0, regions = 1;
    const float* p_o = nullptr;
    const float2* p_ml = nullptr;
    {
        const int p = bad ? -1 : prefix_of(k.prefix, b);
        if (p >= 0) {
            bool no;
            const Group g = group_at(k, p, &no);
            const int f = (b - g.first) * k.R + x;
            if (g.items > 0) {
                const int blocks = (g.rows + 255) / 256;
                const int i = h * blocks + (f >> 8);
                const long long at = us + i * g.item_units() + kItemUnits;
                const long long G = working_blocks(U, a.prefix_grid);
                const int c0 = block_of(at, U, G);
                np = block_of(at + (long long)(g.tiles - 1) * kTileUnits, U, G) - c0 + 1;
                regions = g.rows > 128 ? 1 : 2;
                const int64_t place = (int64_t(item) + i + c0) * 256 + (f & 255);
                p_o = k.state + place * D;
                p_ml = k.state_ml + place;
            }
        }
    }
    const int mine = np * regions;
    const int seg_rows = 8 * a.row_tiles;                // rows of a segment's slot
    const int ms = x / kSegmentRows, xr = x - ms * kSegmentRows;
    const int hm = h * a.MS + ms;
    const int seg = b * a.per_req + hm;
    const int len = granules(b);
    const int64_t units = total + int64_t(k.B) * a.per_req;
    const int64_t grid = suffix_blocks(units, a.suffix_grid);
    const int64_t u0 = ahead + int64_t(hm) * len + (seg + 1);
    const int64_t first = block_of_unit(u0, units, grid);
    const int ns = int(block_of_unit(u0 + len - 1, units, grid) - first) + 1;
    const int slot = suffix_slot_floats(D, a.row_tiles);
    const float* s_at = a.suffix_state + (int64_t(seg) + first) * slot;
    const int pieces = mine + ns;
    auto state_of = [&](int t) -> const float* {
        if (t < mine) {
            const int c = regions == 2 ? t >> 1 : t;
            return p_o + (int64_t(c) * 256 + (regions == 2 ? (t & 1) * 128 : 0)) * D;
        }
        return s_at + int64_t(t - mine) * slot + xr * D;
    };
    auto ml_of = [&](int t) -> const float2* {
        if (t < mine) {
            const int c = regions == 2 ? t >> 1 : t;
            return p_ml + int64_t(c) * 256 + (regions == 2 ? (t & 1) * 128 : 0);
        }
        return reinterpret_cast<const float2*>(s_at + int64_t(t - mine) * slot + seg_rows * D + 2 * xr);
    };

    grid_dependency_wait();
    // ---- the largest maximum, each piece's factor, the sum
    float top = -INFINITY;
    for (int t = threadIdx.x; t < pieces; t += kMergeThreads)
        top = fmaxf(top, __ldcg(ml_of(t)).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        red[0][warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float sum = 0.f;
    for (int t = threadIdx.x; t < pieces; t += kMergeThreads) {
        const float2 v = __ldcg(ml_of(t));
        const float w = v.x == -INFINITY ? 0.f : fast_exp2(v.x - top);
        weights[t] = w;
        sum += w * v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0)
        red[1][warp] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    // ---- the outputs: warp w takes pieces w, w + 4, ...
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int t = warp; t < pieces; t += kMergeThreads / 32) {
        const float w = weights[t];
        if (w > 0.f) {                                   // nothing seen: the state was not written
            if constexpr (D == 128) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(state_of(t)) + lane);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(state_of(t)) + lane);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
            }
        }
    }
    sums[warp][lane] = o;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kMergeThreads / 32; ++w) {
            const float4 v = sums[w][lane];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        const float inv = sum > 0.f ? a.out_scale / sum : 0.f;
        uint16_t* dst = a.out + ((int64_t(b) * k.H_q + h * k.G) * k.L + x) * D;
        if constexpr (D == 128)
            reinterpret_cast<uint2*>(dst)[lane] =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        else
            reinterpret_cast<uint32_t*>(dst)[lane] = pack_bf16x2(o.x * inv, o.y * inv);
    }
}

}  // namespace

size_t prefix_smem_bytes(int D, int count)
{
    return size_t(D == 64 ? Layout<64>::kGroups : Layout<128>::kGroups) + size_t(count) * sizeof(Group) + 1024;
}

size_t prefix_state_bytes(const pa_shape& s, int count, int grid, size_t* ml_off)
{
    const int64_t R = int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len;
    const int64_t items = s.num_kv_heads * (int64_t(s.batch) * R / 256 + count);
    const size_t slots = size_t(items + grid);
    *ml_off = slots * 256 * size_t(s.head_dim) * sizeof(float);
    return *ml_off + slots * 256 * sizeof(float2);
}

cudaError_t launch_prefix(const CUtensorMap& key_map, const CUtensorMap& value_map, const PrefixKernelArgs& a,
                          int D, int grid, int device, cudaStream_t stream)
{
    using Kernel = void (*)(CUtensorMap, CUtensorMap, PrefixKernelArgs);
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev][2];
    static std::atomic<int> regs_ok[kMaxDev][2];
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    const int which = D == 64 ? 0 : 1;
    const Kernel kernel = D == 64 ? prefix_kernel<64> : prefix_kernel<128>;
    const void* fn = reinterpret_cast<const void*>(kernel);
    // setmaxnreg draws on the registers that the block was launched with
    int rk = regs_ok[device][which].load(std::memory_order_relaxed);
    if (rk == 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, fn);
        if (e != cudaSuccess)
            return e;
        rk = fa.numRegs >= kRegsProducer && fa.numRegs <= kRegsSoftmax &&
                     128 * kRegsProducer + 256 * kRegsSoftmax <= kThreads * fa.numRegs
                 ? 1
                 : 2;
        regs_ok[device][which].store(rk, std::memory_order_relaxed);
    }
    if (rk != 1)
        return cudaErrorNotSupported;
    cudaError_t e = raise_smem_limit(fn, &raised[device][which]);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = prefix_smem_bytes(D, a.prefix.count);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, key_map, value_map, a);
}

cudaError_t launch_prefix_merge(const PrefixMergeArgs& a, int D, cudaStream_t stream)
{
    const PrefixKernelArgs& k = a.prefix_args;
    const int64_t blocks = int64_t(k.B) * k.H_kv * k.R;
    if (blocks <= 0 || blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = size_t(2 * a.prefix_grid + a.suffix_grid + 2) * sizeof(float);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, D == 64 ? prefix_merge_kernel<64> : prefix_merge_kernel<128>, a);
}

}  // namespace pa
