// Internal declarations shared by the library's translation units (host
// launchers and kernel argument blocks). Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pagedattn.h"

namespace pa {

// Device error bits (same values as the PA_DEVERR_* macros of the header).
constexpr unsigned PA_DEVERR_PAGE_ID_BIT = 0x1u;
constexpr unsigned PA_DEVERR_SLOT_BIT = 0x2u;
constexpr unsigned PA_DEVERR_CONTEXT_LEN_BIT = 0x4u;
constexpr unsigned PA_DEVERR_TIMEOUT_BIT = 0x8u;
constexpr unsigned PA_DEVERR_POSITION_BIT = 0x10u;
constexpr unsigned PA_DEVERR_PREFIX_BIT = 0x20u;

// Longest a kernel waits for one pipeline phase before giving up, and the
// limit of every later wait of a block that already gave up once.
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint64_t kShortWaitLimitNs = 20000000ull;

// The current device's properties, looked up once.
struct DeviceInfo {
    bool ready = false;
    int id = 0;
    int sm_count = 0;
    int max_smem_optin = 0;
    unsigned* err = nullptr;  // device address of the error word
};
pa_status device_info(DeviceInfo** out);

// Raises a kernel's limit of dynamic shared memory, once per device (*raised), to all
// that a block can have there: the same number whatever the call's batch, so that host
// threads whose first calls meet do not lower each other's.
cudaError_t raise_smem_limit(const void* kernel, std::atomic<bool>* raised);

// Division of 0 .. 2^31 - 1 by a fixed number: with s = ceil(log2 d), m = floor(2^32 (2^s - d)
// / d) + 1 the quotient is (umulhi(m, n) + n) >> s.
struct FixedDivisor {
    uint32_t mul;
    int32_t shift;
    void set(int32_t d)
    {
        shift = 0;
        while ((int64_t(1) << shift) < d)
            ++shift;
        mul = uint32_t((((uint64_t(1) << shift) - uint64_t(d)) << 32) / uint64_t(d) + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int of(int n) const { return int((__umulhi(mul, uint32_t(n)) + uint32_t(n)) >> shift); }
#endif
};

// ---------------------------------------------------------------------------
// Write path

struct AppendArgs {
    const uint16_t* key;          // [B, H_kv, L_new, D]
    const uint16_t* value;
    uint16_t* key_pages;          // [P, H_kv, ps, D]
    uint16_t* value_pages;
    const int32_t* slot_mapping;  // [B, L_new]
    unsigned* err;
    int32_t B, L_new, H_kv, D, ps, num_pages;
    int32_t fp8;                  // 1: the pages hold e4m3 codes (one byte each)
    float k_scale, v_scale;       // e4m3 pages: code = e4m3(x / scale)
};

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);

// Norms, rotation and append of a fused QKV projection's rows.
struct NormRopeArgs {
    const uint16_t* qkv;          // row of token (b, i) at b * batch_stride + i * token_stride:
    int64_t batch_stride;         // H_q query heads, H_kv key heads, H_kv value heads of D
    int64_t token_stride;
    const uint16_t* q_weight;     // [D] bf16, or null: no norm
    const uint16_t* k_weight;
    const float* cos_sin;         // [table_len, rotary_dim]: cos of the angles, then sin
    const int32_t* positions;     // [B, L]
    uint16_t* query;              // [B, H_q, L, D]
    uint16_t* key_pages;          // [P, H_kv, ps, D] bf16, or e4m3 codes
    uint16_t* value_pages;
    const int32_t* slot_mapping;  // [B, L]
    unsigned* err;
    int32_t B, L, H_q, H_kv, D, ps_shift, num_pages;
    int32_t rotary_dim, table_len, interleaved;
    int32_t q_groups, kv_groups;  // set by the launcher: lane groups per token and kind
    int32_t fp8;
    float eps, k_scale, v_scale;
};

cudaError_t launch_norm_rope_append(NormRopeArgs a, cudaStream_t stream);

// Eviction: the slots to keep of every (request, KV head), moved to the front
// of the destination table's pages.
struct EvictArgs {
    void* key_pages;              // [P, H_kv, ps, D], row_bytes each row
    void* value_pages;
    float* weight_pages;          // [P, H_kv, ps]
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* dst_table;     // [B, dst_max_pages]; the block table: in place
    const int32_t* context_lens;  // [B]
    int32_t* kept;                // [B, H_kv, keep]
    int32_t* new_lens;            // [B]
    unsigned* err;
    int32_t B, H_kv, row_bytes, ps_shift, num_pages, max_pages, dst_max_pages;
    int32_t keep, sinks, recent;
    int32_t slices, chunks, chunk_rows;   // set by the launcher: column slices of a row, chunks of rows
};

cudaError_t launch_evict(EvictArgs a, int device, int sm_count, cudaStream_t stream);

struct GatherArgs {
    const uint16_t* key_pages;    // [P, H_kv, ps, D]
    const uint16_t* value_pages;
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    uint16_t* key_dense;          // [B, H_kv, dense_len, D]
    uint16_t* value_dense;
    unsigned* err;
    int32_t B, H_kv, D, ps, num_pages, max_pages, dense_len;
};

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream);

// 4-bit pools (pa_q4.cuh): the quantising append (AppendArgs, pages of 80-byte rows,
// D 128), and the read-back of every request's rows as bf16 (kind; bf16 pools also with
// head_dim 64: rows of D elements then). Row t of (request b,
// KV head h) goes to element b * batch_stride + h * head_stride + (t / 128) * block_stride
// + (t % 128) * D: dense rows, or pages of 128 tokens with a table (table_out
// [B, copy_pages], page b * copy_pages + t / 128; rows of a bad page are zeros there).
constexpr int kCopyPageRows = 128;
struct PageReadArgs {
    const uint8_t* key_pages;     // [P, H_kv, ps, row bytes]
    const uint8_t* value_pages;
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    uint16_t* key_out;
    uint16_t* value_out;
    int32_t* table_out;           // null: dense rows
    unsigned* err;
    int64_t batch_stride, head_stride, block_stride;
    int32_t B, H_kv, ps, num_pages, max_pages;
    int32_t max_len;              // rows a request has room for
    int32_t copy_pages;
    int32_t f16_values;           // the values leave as f16 (4-bit rows; else bf16)
    int32_t chunks;               // set by the launcher, like the divisors
    FixedDivisor by_chunks, by_H;
};
cudaError_t launch_append_q4(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_read_pages(PageReadArgs a, int kind, int D, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Split-KV attention (decode schedule)

// Work decomposition: the G * L query rows of a (request b, KV head h) are
// cut into tiles of 16 rows, and a "segment" is (b, h, group of TG
// consecutive row tiles); its keys are cut into granules of kDecodeTokens
// tokens, and every K/V granule loaded serves all TG tiles. All granules of
// all segments form one stream that the grid splits evenly; a segment that
// straddles blocks leaves one partial state per block, merged by a second,
// small kernel.
constexpr int kDecodeTokens = 64;
constexpr int kDecodeRows = 16;

// At most this many (request x KV head x 16-row tile) per call.
constexpr int64_t kMaxSegments = 65536;

// Row tiles per segment and segment count of a decode call: one tile per
// segment when the rows fit one tile (and always on e4m3 pools), otherwise
// 2 tiles (2 tiles of rows) or 4 (3 or more; a group of 3 tiles leaves the
// fourth slot empty).
struct DecodePlan {
    int32_t MT;      // 16-row tiles per (request, KV head): ceil(G * L / 16)
    int32_t TG;      // row tiles per segment: 1, 2 or 4
    int32_t MS;      // segments per (request, KV head): ceil(MT / TG)
    int64_t nseg;    // B * H_kv * MS
};
DecodePlan decode_plan(const pa_shape& s, bool fp8);

// What a decode kernel attends to and leaves: everything; a sliding window and
// the first keys; everything, with the scores and row states kept.
// The few-row kernel also: the keys behind a shared prefix, states left as rows.
enum DecodeMode : int { kFull = 0, kWindow = 1, kScores = 2, kDecodeModes = 3, kSuffix = 3 };

// What a pool's rows hold.
enum PoolKind : int { kBf16Pool = 0, kE4m3Pool = 1, kQ4Pool = 2 };

// Query rows of a segment of the few-row kernel, where a call has more.
constexpr int kSegmentRows = 16;

// The prefixes that requests of a batch share (pa_prefix.cuh).
struct PrefixArgs {
    const int32_t* table;         // [count, pages]
    const int32_t* lens;          // [count]
    const int32_t* starts;        // [count + 1]
    int32_t count, pages;
    int32_t cap;                  // longest prefix
};

struct DecodeArgs {
    const uint16_t* q;            // [B, H_q, L, D]
    uint16_t* out;                // [B, H_q, L, D]
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    float* partials;              // [slots][TG][m[16], l[16], acc[16][D]]
    unsigned* err;
    int32_t B, H_q, H_kv, L, D, ps, max_pages, num_pages;
    int32_t G;          // H_q / H_kv
    int32_t R;          // G * L query rows per (request, KV head)
    int32_t MS;         // segments per (request, KV head): ceil(ceil(R / 16) / TG)
    int32_t TG;         // 16-row tiles per segment (1, 2 or 4); tile t of segment
                        // ms holds rows [16 (ms TG + t), 16 (ms TG + t) + 16) of R
    int32_t box_rows;   // rows per TMA box: min(ps, 64); the few-row kernel min(ps, its tile of 16 or 32)
    int32_t swz;        // 7: 128B-swizzled stage layout (box_rows >= 8); 0: linear
    int32_t whole_segments;  // 1: every block takes whole segments (no partials)
    int32_t piece_units;     // split weight of a piece beyond its granules (set by
                             // the launcher for the merge pass)
    int32_t dense;      // 1: K/V are dense [B, H_kv, ps, D] (request b is page b;
                        // block_table is not read)
    float scale_log2;   // scale * log2(e) (times k_scale for e4m3 pages)
    int32_t causal;
    int32_t fp8;        // 1: K/V pages hold e4m3 codes (head_dim 128)
    float v_scale;      // e4m3 pages: the value scale (1 otherwise)
    int32_t mode;       // DecodeMode
    int32_t window;     // kWindow: keys a row sees, its own among them
    int32_t sinks;      // kWindow: first keys that stay visible
    float* scores;      // kScores: [B * H_kv][R][score_stride], log2 domain
    float2* row_state;  // kScores: [B * H_kv][R] (max, sum)
    int64_t score_stride;      // a multiple of 64, at least score_cap
    int32_t score_cap;         // kScores: longest context
    int32_t ps_shift;   // the few-row kernel: log2 of the page size
    const uint8_t* key_rows;      // 4-bit pools
    const uint8_t* value_rows;
    PrefixArgs prefix;            // kSuffix
    int2* note_segment;           // kSuffix: for the merge (PrefixMergeArgs)
    int32_t debug_unset_wait;  // test support: block 0 first waits on a barrier
                               // that nothing arrives at (times out, flags)
};

size_t decode_smem_bytes(int D, int B, bool fp8 = false, int TG = 1);   // dynamic
size_t decode_static_smem_bytes(bool fp8);
int decode_max_grid(int sm_count);
size_t decode_workspace_bytes(int64_t nseg, int grid_max, int D, int TG);
cudaError_t launch_decode(const CUtensorMap& key_map, const CUtensorMap& value_map,
                          const CUtensorMap& q_map, const DecodeArgs& a, int grid, int device,
                          cudaStream_t stream);

// The few-row kernel: whether it takes a window or weight call (at most 16 rows per
// request and KV head) on a device with max_smem bytes of shared memory a block;
// whether the modes that cut more rows into segments fit (kFull over 4-bit pools,
// kSuffix); the keys per TMA box (DecodeArgs::box_rows); its workspace; its blocks
// (granule_bound: an upper bound of the 4-tile granules, 0 unknown) and the launch.
bool decode_rows_takes(const pa_shape& s, int max_smem);
bool decode_rows_fits(const pa_shape& s, int kind, int mode, int max_smem);
int decode_rows_box(const pa_shape& s, int kind, int page_size);
size_t decode_rows_workspace_bytes(const pa_shape& s, int kind, int mode, int sm_count);
int decode_rows_tile(const pa_shape& s, int kind);     // keys of a tile
int decode_rows_row_tiles(const pa_shape& s);          // 8-row tiles of a segment
int decode_rows_launch_grid(const pa_shape& s, int kind, int mode, int64_t granule_bound, int sm_count);
cudaError_t launch_decode_rows(const CUtensorMap& key_map, const CUtensorMap& value_map, DecodeArgs a,
                               const pa_shape& s, int kind, int grid, void* workspace, int device,
                               cudaStream_t stream);

// Decode behind shared prefixes: the prefixes' part for all their requests' rows, and
// the merge of it with the few-row kernel's (kSuffix).
struct PrefixKernelArgs {
    const uint16_t* q;            // [B, H_q, L, D]
    const int32_t* context_lens;  // [B]
    float* state;                 // [slot][256 rows][D]
    float2* state_ml;             // [slot][256] (max, sum)
    unsigned* err;
    PrefixArgs prefix;            // table of the pages that the maps lead to
    int32_t B, H_q, H_kv, L, G, R;
    int32_t ps, num_pages;        // of those pages
    int32_t box_rows;             // min(ps, 128), at least 8
    int32_t block_ps, max_pages;  // of the requests' own tables
    const uint8_t* key_rows;      // e4m3 and 4-bit pools
    const uint8_t* value_rows;
    int32_t ps_shift;             // log2 of ps
    FixedDivisor by_R, by_L, by_H;   // by_H: H_kv
    int4* note_row;               // [B * H_kv * R] its first state in the prefix, states, place in
                                  // them, 1: both halves of a state hold the rows
    void* more_pieces;            // [grid][most_items]
    int32_t most_items;
    float scale_log2;
};
struct PrefixMergeArgs {
    PrefixKernelArgs prefix_args;
    const float* suffix_state;    // [slot][row_tiles * 8 * (D + 2)]
    uint16_t* out;                // [B, H_q, L, D]
    float out_scale;
    const int2* note_segment;     // [B * H_kv * MS] first and last block
    int32_t MS, row_tiles;        // of the few-row kernel
    int32_t share;                // set by the launcher: warps a row
};
constexpr int kMaxPrefixes = 256;      // their tables lie in shared memory
// A block's pieces of items that lie in shared memory; an item's units of work.
constexpr int kPrefixMaxPieces = 64;
inline int64_t prefix_item_units(int64_t tiles) { return tiles * 4 + 16; }
size_t prefix_smem_bytes(int D, int kind, int count);
// The workspace of the states of `items` items, and where (m, l) and the pieces behind
// kPrefixMaxPieces start in it.
size_t prefix_state_bytes(const pa_shape& s, int64_t items, int grid, size_t* ml_off, size_t* pieces_off);
// What can fail before the launch: the limits of the device. cudaErrorNotSupported: a
// build whose registers the kernel cannot split.
cudaError_t prepare_prefix(int D, int kind, int device);
cudaError_t launch_prefix(const CUtensorMap& key_map, const CUtensorMap& value_map, const PrefixKernelArgs& a,
                          int D, int kind, int grid, cudaStream_t stream);
cudaError_t launch_prefix_merge(PrefixMergeArgs a, int D, int sm_count, cudaStream_t stream);

// Accumulation of attention weights: weight_pages[slot of j] = decay * old (0
// for the L newest positions, or where decay is 0) + sum over the R rows of
// 2^(score - max) / sum.
struct WeightArgs {
    const float* scores;          // as in DecodeArgs
    const float2* row_state;
    float* weight_pages;          // [P, H_kv, ps]
    const int32_t* block_table;
    const int32_t* context_lens;
    int64_t score_stride;
    int32_t B, H_kv, R, L, ps_shift, max_pages, num_pages, score_cap;
    int32_t chunks;               // set by the launcher: blocks per (request, KV head)
    float decay;
};
cudaError_t launch_accumulate_weights(WeightArgs a, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Prefill on the 5th-generation tensor cores (D = 128, page_size >= 8)

struct PrefillArgs {
    uint16_t* out;                // [B, H_q, L, D]
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    unsigned* err;
    int32_t B, H_q, H_kv, L, ps, max_pages, num_pages;
    int32_t G;          // H_q / H_kv
    int32_t n_qtiles;   // ceil(L / 128)
    int32_t box_rows;   // rows per K/V TMA box: min(ps, 128)
    float scale_log2;
    int32_t causal;
    float out_scale;    // the output is out_scale * softmax . V (e4m3 copies: v_scale)
    int32_t D;          // head_dim: 128 (64 on the pairs kernel only)
    // The pools, read row by row on the pairs kernel when a page holds fewer
    // than 8 tokens (otherwise through the tensor maps).
    const uint16_t* key_pages;    // [P, H_kv, ps, D]
    const uint16_t* value_pages;
    // Pairs kernel, tail pieces (head_dim 128; state == nullptr: none): per
    // donor block slot, part (0: the item's last tiles, 1: its first tiles)
    // and head, O / l in bf16 [16 chunks of 8 columns][128 rows] and (m, l)
    // per row; per slot, head and softmax warp one arrival word (the launch's
    // stamp in the high 32 bits, the arrivals in the low 32).
    uint4* state;                 // [grid][2][2][16][128]
    float2* state_ml;             // [grid][2][2][128]
    unsigned long long* arrive;   // [grid][2][4]
    uint64_t stamp;               // this launch's stamp (never 0)
    int32_t piece_last;           // test setting: receiving blocks run the piece last
    // Pairs kernel: a sliding window of `window` keys (0: none; causal) and the
    // first `sinks` keys.
    int32_t window, sinks;
    int32_t f16_values;           // V holds f16 (head_dim 128, pages of 8 tokens or more, no window)
};

// Prefill over e4m3 pools: bf16 copies of the K/V tokens that some row sees, in
// pages of 128 tokens, P1 a request, and a table of P2 entries a request that leads
// to them: entry p is the copy page of tokens [128 p, 128 p + 128). Without a window
// P1 = P2 and entry p of request b is b * P2 + p. With one, copy page b * P1 + i is
// that of the sinks' i-th 128 tokens, and behind the sinks' pages of the i-th from
// the first token on that some row sees through the window; entries of tokens
// that no row sees are not written.
struct Fp8PagesArgs {
    const uint8_t* key_pages;     // [P, H_kv, ps, 128] e4m3 codes
    const uint8_t* value_pages;
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    uint16_t* key_out;            // [B * P1, H_kv, 128, 128] bf16
    uint16_t* value_out;
    int32_t* table_out;           // [B, P2]
    unsigned* err;
    int32_t B, H_kv, ps, max_pages, num_pages;
    int32_t P2;                   // ceil(max_context_len / 128)
    // A sliding window (0: none, and P1 is not read) over L query rows.
    int32_t window, sinks, L;
    int32_t P1;
};
// Copy pages per request with a sliding window.
int64_t fp8_window_pages(int64_t max_context_len, int64_t window, int64_t sinks, int64_t L);
int64_t fp8_copy_pages(int64_t max_context_len);
cudaError_t launch_fp8_pages_to_bf16(const Fp8PagesArgs& a, cudaStream_t stream);

// Stamps for the publish flags of kernels that hand partial states between
// blocks: distinct for every launch of this process, the first one
// seeded from a clock reading so that flags left in a workspace by an earlier
// process are not mistaken for this launch's. Never 0; 48 bits.
uint64_t next_launch_stamp();

// Prefill with the K/V tiles of all (request, head pair, query tile) items
// split evenly over a persistent grid (one block per SM, all resident); an
// item cut by a block boundary is finished by the block that holds its first
// tiles, which merges the states the later pieces left in the workspace.
struct SplitPrefillArgs {
    uint16_t* out;                // [B, H_q, L, 128]
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* context_lens;  // [B]
    unsigned* err;
    float* state;                 // [grid][head 2][32][128][4]
    float2* state_ml;             // [grid][head 2][128] (m, l)
    unsigned long long* flags;    // [grid][head 2][4 warps]: stamp when written
    uint64_t stamp;               // this launch's stamp (never 0)
    int32_t B, H_q, H_kv, L, ps, max_pages, num_pages;
    int32_t G;          // H_q / H_kv (>= 2; odd: the last pair repeats its head)
    int32_t n_qtiles;   // ceil(L / 128)
    int32_t box_rows;   // rows per K/V TMA box: min(ps, 128)
    float scale_log2;
    int32_t causal;
    float out_scale;    // the output is out_scale * softmax . V (e4m3 copies: v_scale)
    int32_t window, sinks;   // window > 0: a sliding window, first keys that stay visible
    int32_t f16_values;      // V holds f16 (no window)
};

size_t prefill_split_smem_bytes();
size_t prefill_split_workspace_bytes(int grid);
cudaError_t launch_prefill_split(const CUtensorMap& q_map, const CUtensorMap& key_map,
                                 const CUtensorMap& value_map, SplitPrefillArgs a, int grid,
                                 void* workspace, int device, cudaStream_t stream);

size_t prefill_smem_bytes();
size_t prefill_pairs_smem_bytes(int D);
// Workspace of the pairs kernel's tail pieces on a grid of `grid` blocks.
size_t prefill_pairs_workspace_bytes(int grid);
// out_map: the output as a 3-D bf16 tensor {D, L, B * H_q}, boxes of 64
// columns x 32 rows, 128-byte swizzle (the kernel stores through it).
// grid_cap: blocks at most (the SM count). workspace (optional, 256-byte
// aligned, any contents): room for tail pieces (prefill_pairs_workspace_bytes
// of the grid); without it, whole items only.
cudaError_t launch_prefill_pairs(const CUtensorMap& q_map, const CUtensorMap& key_map,
                                 const CUtensorMap& value_map, const CUtensorMap& out_map,
                                 const PrefillArgs& a, int device, int grid_cap, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream);
cudaError_t launch_prefill(const CUtensorMap& q_map, const CUtensorMap& key_map,
                           const CUtensorMap& value_map, const PrefillArgs& a, int device,
                           cudaStream_t stream);

// Host-side checks of a decode call (everything pa_decode rejects before
// launching, except the workspace), and its number of segments.
pa_status validate_decode(const void* query, const void* key_pages, const void* value_pages,
                          const int32_t* block_table, const int32_t* context_lens,
                          int32_t page_size, float scale, const void* out, const pa_shape& s);
int64_t decode_segment_count(const pa_shape& s);

}  // namespace pa
