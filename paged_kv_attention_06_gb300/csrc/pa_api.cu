// C ABI of the paged-attention library: argument checks, tensor-map set-up,
// the dispatch rule, and the device error word. No entry point allocates
// device memory; every launch goes on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <initializer_list>
#include <mutex>

#include "../../include/pagedattn.h"
#include "../../include/pagedattn_test.h"
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

// Device error word: kernels OR PA_DEVERR_* bits into it; pa_get_device_error
// reads and clears it. One copy per device that loads the library.
__device__ unsigned int g_device_error;

uint64_t next_launch_stamp()
{
    static std::atomic<uint64_t> stamp{0};
    if (stamp.load(std::memory_order_relaxed) == 0) {
        const uint64_t seed = uint64_t(
            std::chrono::steady_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ull;
        uint64_t expected = 0;
        stamp.compare_exchange_strong(expected, (seed >> 16) | 1ull);
    }
    uint64_t st = stamp.fetch_add(1, std::memory_order_relaxed) & ((uint64_t(1) << 48) - 1);
    return st == 0 ? 1 : st;
}

namespace {

constexpr int kMaxDevices = 64;

std::mutex g_mutex;
thread_local bool t_arm_unset_wait = false;  // test support, see pa_debug_arm_wait_timeout
thread_local int t_prefill_variant = 0;      // see pa_debug_prefill_variant
DeviceInfo g_devices[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

}  // namespace

pa_status device_info(DeviceInfo** out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return PA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceInfo& d = g_devices[dev];
    if (!d.ready) {
        int sms = 0, smem = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
                cudaSuccess)
            return PA_ERR_CUDA;
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess)
            return PA_ERR_CUDA;
        d.id = dev;
        d.sm_count = sms;
        d.max_smem_optin = smem;
        d.err = static_cast<unsigned*>(p);
        d.ready = true;
    }
    *out = &d;
    return PA_OK;
}

cudaError_t raise_smem_limit(const void* kernel, std::atomic<bool>* raised)
{
    if (raised->load(std::memory_order_relaxed))
        return cudaSuccess;
    DeviceInfo* dev;
    if (device_info(&dev) != PA_OK)
        return cudaErrorInvalidDevice;
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 dev->max_smem_optin - int(fa.sharedSizeBytes));
    if (e == cudaSuccess)
        raised->store(true, std::memory_order_relaxed);
    return e;
}

namespace {

pa_status get_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_encode) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !p)
            return PA_ERR_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    *fn = g_encode;
    return PA_OK;
}

// Encodes a tensor map. The driver wants a current context: a host thread whose first
// CUDA call this is has none until the runtime binds its device's.
template <typename... Args>
pa_status encode_map(Args... args)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const pa_status st = get_encoder(&enc);
    if (st != PA_OK)
        return st;
    CUresult r = enc(args...);
    if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess)
            return PA_ERR_CUDA;
        r = enc(args...);
    }
    return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool pow2_in(int v, int lo, int hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }

// Checks shared by the attention entry points.
pa_status check_attention(const void* query, const void* key_pages, const void* value_pages,
                          const int32_t* block_table, const int32_t* context_lens,
                          int32_t page_size, float scale, const void* out, const pa_shape& s)
{
    if (!query || !key_pages || !value_pages || !block_table || !context_lens || !out)
        return PA_ERR_INVALID_ARG;
    if (s.batch <= 0 || s.num_q_heads <= 0 || s.num_kv_heads <= 0 || s.q_len <= 0 ||
        s.num_pages <= 0 || s.max_pages <= 0 || s.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query) || !aligned16(key_pages) || !aligned16(value_pages) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    if (s.head_dim != 64 && s.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    if (s.num_q_heads % s.num_kv_heads != 0)
        return PA_ERR_UNSUPPORTED;
    if (!pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    // TMA row coordinates and in-kernel page arithmetic are 32-bit.
    if (int64_t(s.num_pages) * s.num_kv_heads * page_size >= (int64_t(1) << 31))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(s.max_pages) * page_size >= (int64_t(1) << 30))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Recently encoded tensor maps of this host thread (a map depends only on
// the pool's address and shape).
struct MapCacheEntry {
    CUtensorMap map;
    const void* pool;
    uint64_t rows;
    int32_t D, ps;
    int box_rows;
    bool fp8;
    bool valid;
};
constexpr int kMapCache = 8;
thread_local MapCacheEntry t_map_cache[kMapCache];
thread_local int t_map_next = 0;

pa_status encode_pool_map_uncached(CUtensorMap* map, const void* pool, const pa_shape& s,
                                   int32_t ps, bool fp8, int box_rows);

// 2-D view of a page pool: rows = P * H_kv * page_size, columns = D (bf16
// elements, or e4m3 codes of one byte when fp8).
pa_status encode_pool_map(CUtensorMap* map, const void* pool, const pa_shape& s, int32_t ps,
                          bool fp8 = false, int box_rows = 0)
{
    if (box_rows == 0)
        box_rows = ps < kDecodeTokens ? ps : kDecodeTokens;
    const uint64_t rows = uint64_t(s.num_pages) * s.num_kv_heads * ps;
    for (int i = 0; i < kMapCache; ++i) {
        const MapCacheEntry& e = t_map_cache[i];
        if (e.valid && e.pool == pool && e.rows == rows && e.D == s.head_dim && e.ps == ps &&
            e.fp8 == fp8 && e.box_rows == box_rows) {
            *map = e.map;
            return PA_OK;
        }
    }
    pa_status st = encode_pool_map_uncached(map, pool, s, ps, fp8, box_rows);
    if (st == PA_OK) {
        MapCacheEntry& e = t_map_cache[t_map_next];
        t_map_next = (t_map_next + 1) % kMapCache;
        e.map = *map;
        e.pool = pool;
        e.rows = rows;
        e.D = s.head_dim;
        e.ps = ps;
        e.fp8 = fp8;
        e.box_rows = box_rows;
        e.valid = true;
    }
    return st;
}

pa_status encode_pool_map_uncached(CUtensorMap* map, const void* pool, const pa_shape& s,
                                   int32_t ps, bool fp8, int box_rows)
{
    const cuuint64_t dims[2] = {cuuint64_t(s.head_dim),
                                cuuint64_t(s.num_pages) * s.num_kv_heads * ps};
    const cuuint64_t strides[1] = {cuuint64_t(s.head_dim) * (fp8 ? 1 : 2)};
    // a box row is 128 bytes: 64 bf16 or 128 e4m3 codes
    const cuuint32_t box[2] = {fp8 ? 128u : 64u, cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    // Boxes of 8+ rows land on 1024-byte boundaries and use the 128-byte
    // swizzle; smaller pages use a linear layout (their destinations are only
    // 128-byte aligned).
    const CUtensorMapSwizzle swz =
        box_rows >= 8 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
    return encode_map(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                     const_cast<void*>(pool), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// 2-D bf16 tensor map over `rows` rows of `cols` columns, boxes of 64 columns
// x box_rows rows, 128-byte swizzle (queries of both kernels, prefill K/V).
pa_status encode_rows_map(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows,
                          uint32_t cols = 128)
{
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(cols) * 2};
    const cuuint32_t box[2] = {64u, box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// 3-D bf16 tensor map over the attention output [B * H_q, L, cols]: boxes of
// 64 columns x 32 rows of one (request, head), 128-byte swizzle (the pairs
// prefill kernel's output stores; rows past L are outside the map).
pa_status encode_out_map(CUtensorMap* map, void* base, uint64_t heads, uint64_t L, uint32_t cols)
{
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(L), cuuint64_t(heads)};
    const cuuint64_t strides[2] = {cuuint64_t(cols) * 2, cuuint64_t(cols) * 2 * L};
    const cuuint32_t box[3] = {64u, 32u, 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// (request, pair of query heads of one KV group, 128-row query tile) items of a
// prefill: ceil(G / 2) pairs per group (an odd group's last pair repeats its
// last head).
int64_t prefill_pair_items(const pa_shape& s)
{
    const int g = s.num_kv_heads > 0 ? s.num_q_heads / s.num_kv_heads : 0;
    return int64_t(s.batch) * ((int64_t(s.q_len) + 127) / 128) * s.num_kv_heads * ((g + 1) / 2);
}

// Workspace the split prefill kernel needs for this shape on this device, or
// 0 when the shape takes another prefill kernel (head_dim 64, pages of fewer
// than 8 tokens, one query head per KV group, or shared memory too small).
size_t split_prefill_need(const pa_shape& s, int32_t page_size, const DeviceInfo* dev)
{
    if (s.head_dim != 128 || page_size < 8 || s.num_kv_heads <= 0 ||
        s.num_q_heads % s.num_kv_heads != 0 || s.num_q_heads / s.num_kv_heads < 2)
        return 0;
    if (prefill_split_smem_bytes() > size_t(dev->max_smem_optin))
        return 0;
    // the same workspace serves the pairs kernel's tail pieces
    const size_t split = prefill_split_workspace_bytes(dev->sm_count);
    const size_t pieces = prefill_pairs_workspace_bytes(dev->sm_count);
    return split > pieces ? split : pieces;
}

// The split kernel. cudaErrorNotSupported: its register split is not available, or
// not every block could be resident (another client holds SMs); the other
// kernels take the call then.
cudaError_t run_split(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                      const PrefillArgs& a, const DeviceInfo* dev, int grid, void* workspace,
                      cudaStream_t stream)
{
    SplitPrefillArgs sa;
    memset(&sa, 0, sizeof sa);
    sa.out = a.out;
    sa.block_table = a.block_table;
    sa.context_lens = a.context_lens;
    sa.err = a.err;
    sa.B = a.B;
    sa.H_q = a.H_q;
    sa.H_kv = a.H_kv;
    sa.L = a.L;
    sa.ps = a.ps;
    sa.max_pages = a.max_pages;
    sa.num_pages = a.num_pages;
    sa.G = a.G;
    sa.n_qtiles = a.n_qtiles;
    sa.box_rows = a.box_rows;
    sa.scale_log2 = a.scale_log2;
    sa.causal = a.causal;
    sa.out_scale = a.out_scale;
    sa.window = a.window;
    sa.sinks = a.sinks;
    sa.f16_values = a.f16_values;
    // An error the caller left pending is not ours to clear: note it, so
    // that only a refused cooperative launch of this call is cleared.
    const bool pending = cudaPeekAtLastError() != cudaSuccess;
    const cudaError_t e = launch_prefill_split(qmap, kmap, vmap, sa, grid, workspace,
                                               dev->id, stream);
    if (e != cudaErrorCooperativeLaunchTooLarge)
        return e;
    if (!pending)
        (void)cudaGetLastError();
    return cudaErrorNotSupported;
}

// Prefill on tcgen05 (D = 128 or 64; pages of fewer than 8 tokens on the
// pairs kernel, whose loaders then copy K/V row by row). With a workspace of at least split_prefill_need
// bytes: the split kernel (K/V tiles spread evenly over one block per SM);
// otherwise the persistent pairs kernel (whole (request, head pair, 128-row
// query tile) items) or one block per (request, query head, query tile).
pa_status run_prefill_tc(const void* query, const void* key_pages, const void* value_pages,
                         const int32_t* block_table, const int32_t* context_lens,
                         int32_t page_size, float scale, int causal, void* out,
                         const pa_shape& s, cudaStream_t stream, void* workspace = nullptr,
                         size_t workspace_bytes = 0, float out_scale = 1.f,
                         void* piece_ws = nullptr, size_t piece_ws_bytes = 0, bool f16_values = false)
{
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    const size_t split_need = split_prefill_need(s, page_size, dev);
    const bool split = t_prefill_variant == 0 && workspace && split_need > 0 &&
                       workspace_bytes >= split_need &&
                       (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0;
    // Two query heads of one KV group per block when the group has at least
    // two (an odd group's last pair repeats its last head), unless the one-head
    // kernel is requested. An odd group with fewer pair items than SMs takes
    // the one-head kernel, whose more numerous blocks fill the GPU better
    // (group of 7, one 512-row chunk after a 16k prefix: 209.6 against 219.8
    // us; with 256 pair items the pairs kernel is 22-33 % faster).
    const int g = s.num_q_heads / s.num_kv_heads;
    const int64_t pair_items = prefill_pair_items(s);
    // Only the pairs kernel has the 64-column form and the row-by-row loads of
    // small pages. With one query head per KV group it takes that head twice,
    // as an odd group's last pair.
    const bool d64 = s.head_dim == 64;
    const bool small_pages = page_size < 8;
    bool pairs = d64 || small_pages ||
                 (g >= 2 && t_prefill_variant != 1 &&
                  (g % 2 == 0 || t_prefill_variant >= 2 || pair_items >= dev->sm_count));
    if (pairs && prefill_pairs_smem_bytes(s.head_dim) > size_t(dev->max_smem_optin))
        pairs = false;
    if ((d64 || small_pages) && !pairs)
        return PA_ERR_UNSUPPORTED;
    if (!pairs && prefill_smem_bytes() > size_t(dev->max_smem_optin))
        return PA_ERR_UNSUPPORTED;
    const int64_t n_qtiles = (int64_t(s.q_len) + 127) / 128;
    const int64_t grid = int64_t(s.batch) * s.num_q_heads * n_qtiles;
    const int64_t q_rows = int64_t(s.batch) * s.num_q_heads * s.q_len;
    if (grid >= (int64_t(1) << 31) || q_rows >= (int64_t(1) << 31))
        return PA_ERR_UNSUPPORTED;
    const uint32_t box = uint32_t(page_size < 128 ? page_size : 128);
    CUtensorMap qmap, kmap, vmap;
    const uint64_t kv_rows = uint64_t(s.num_pages) * s.num_kv_heads * page_size;
    const uint32_t cols = uint32_t(s.head_dim);
    CUtensorMap omap;
    if ((st = encode_rows_map(&qmap, query, uint64_t(q_rows), 128u, cols)) != PA_OK ||
        (st = encode_rows_map(&kmap, key_pages, kv_rows, box, cols)) != PA_OK ||
        (st = encode_rows_map(&vmap, value_pages, kv_rows, box, cols)) != PA_OK ||
        (st = encode_out_map(&omap, out, uint64_t(s.batch) * s.num_q_heads, uint64_t(s.q_len), cols)) !=
            PA_OK)
        return st;
    PrefillArgs a;
    memset(&a, 0, sizeof a);
    a.out = static_cast<uint16_t*>(out);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.L = s.q_len;
    a.ps = page_size;
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.G = s.num_q_heads / s.num_kv_heads;
    a.n_qtiles = int32_t(n_qtiles);
    a.box_rows = int32_t(box);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = causal ? 1 : 0;
    a.out_scale = out_scale;
    a.D = s.head_dim;
    a.f16_values = f16_values ? 1 : 0;
    a.key_pages = static_cast<const uint16_t*>(key_pages);
    a.value_pages = static_cast<const uint16_t*>(value_pages);
    a.piece_last = t_prefill_variant == 5 ? 1 : 0;
    if (split) {
        const cudaError_t e = run_split(qmap, kmap, vmap, a, dev, dev->sm_count, workspace, stream);
        if (e != cudaErrorNotSupported)
            return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    // The pairs kernel's tail pieces use the caller's workspace (pa_attention's).
    // Test setting 4: a grid of two thirds of the items, so that small shapes
    // have blocks of one item and of two, and get pieces.
    const bool small_grid = t_prefill_variant == 4 || t_prefill_variant == 5;
    const int grid_cap = small_grid ? int((2 * pair_items + 2) / 3) : dev->sm_count;
    cudaError_t e = pairs ? launch_prefill_pairs(qmap, kmap, vmap, omap, a, dev->id, grid_cap,
                                                 t_prefill_variant == 0 || small_grid ? piece_ws : nullptr,
                                                 piece_ws_bytes, stream)
                          : launch_prefill(qmap, kmap, vmap, a, dev->id, stream);
    if (pairs && e == cudaErrorNotSupported) {   // register split not available
        if (d64 || small_pages)
            return PA_ERR_UNSUPPORTED;
        e = launch_prefill(qmap, kmap, vmap, a, dev->id, stream);   // one head per block
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Blocks of the split kernel for a windowed prefill, or 0: the pairs kernel. With t
// tiles an item, whole items take the time of R t tiles, R = ceil(items / SMs); the
// split kernel that of a block's share of all tiles (two more an item) and about
// ten for what it adds (a launch that overlaps no other, the merges). Measured, 32
// heads on 8, one request, pairs and split in us: 64 items, window 2048 37 and 35,
// 4096 63 and 47, 16384 216 and 122; 96 items, 4096 63 and 60; 128 items, 4096 64
// and 72, 16384 218 and 222; 160 items, 1024 40 and 36, 2048 66 and 50, 4096 117
// and 80; 1024 items, 4096 306 and 358. Blocks of fewer than 8 tiles merge too many
// states (16 items, window 4096: 45 against 40). max_context_len 0: unknown.
int window_split_grid(const pa_shape& s, int32_t page_size, int32_t max_context_len, int32_t window,
                      int32_t sinks, const DeviceInfo* dev)
{
    if (split_prefill_need(s, page_size, dev) == 0)
        return 0;
    const int64_t context = max_context_len > 0 ? max_context_len : int64_t(s.max_pages) * page_size;
    const int64_t keys = std::min(context, int64_t(window) + sinks + 127);
    const int64_t t = (keys + 127) / 128, items = prefill_pair_items(s), sms = dev->sm_count;
    const int64_t tiles = items * (t + 2);
    if (t_prefill_variant == 6)            // test setting: always, in small pieces
        return int(std::max<int64_t>(1, std::min(sms, tiles / 2)));
    const int64_t grid = std::max<int64_t>(1, std::min(sms, tiles / 8));
    const int64_t whole = (items + sms - 1) / sms * t, share = (tiles + grid - 1) / grid;
    return 10 * whole > 11 * (share + 10) ? int(grid) : 0;
}
size_t window_split_need(const pa_shape& s, int32_t page_size, int32_t max_context_len,
                         int32_t window, int32_t sinks, const DeviceInfo* dev)
{
    const int grid = window_split_grid(s, page_size, max_context_len, window, sinks, dev);
    return grid > 0 ? prefill_split_workspace_bytes(grid) : 0;
}

// Prefill with a sliding window: the split kernel where window_split_grid says so
// and the workspace is large enough, otherwise the pairs kernel (every head_dim, page size
// and group size; whole items). PA_ERR_UNSUPPORTED where the register split is not
// available.
pa_status run_prefill_window(const void* query, const void* key_pages, const void* value_pages,
                             const int32_t* block_table, const int32_t* context_lens,
                             int32_t page_size, float scale, int32_t window, int32_t sinks,
                             float out_scale, void* out, const pa_shape& s,
                             int32_t max_context_len, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream)
{
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (prefill_pairs_smem_bytes(s.head_dim) > size_t(dev->max_smem_optin) || t_prefill_variant == 7)
        return PA_ERR_UNSUPPORTED;
    const int64_t n_qtiles = (int64_t(s.q_len) + 127) / 128;
    const int64_t q_rows = int64_t(s.batch) * s.num_q_heads * s.q_len;
    if (int64_t(s.batch) * s.num_q_heads * n_qtiles >= (int64_t(1) << 31) ||
        q_rows >= (int64_t(1) << 31))
        return PA_ERR_UNSUPPORTED;
    const uint32_t box = uint32_t(page_size < 128 ? page_size : 128);
    const uint64_t kv_rows = uint64_t(s.num_pages) * s.num_kv_heads * page_size;
    const uint32_t cols = uint32_t(s.head_dim);
    CUtensorMap qmap, kmap, vmap, omap;
    if ((st = encode_rows_map(&qmap, query, uint64_t(q_rows), 128u, cols)) != PA_OK ||
        (st = encode_rows_map(&kmap, key_pages, kv_rows, box, cols)) != PA_OK ||
        (st = encode_rows_map(&vmap, value_pages, kv_rows, box, cols)) != PA_OK ||
        (st = encode_out_map(&omap, out, uint64_t(s.batch) * s.num_q_heads, uint64_t(s.q_len),
                             cols)) != PA_OK)
        return st;
    PrefillArgs a;
    memset(&a, 0, sizeof a);
    a.out = static_cast<uint16_t*>(out);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.L = s.q_len;
    a.ps = page_size;
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.G = s.num_q_heads / s.num_kv_heads;
    a.n_qtiles = int32_t(n_qtiles);
    a.box_rows = int32_t(box);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = 1;
    a.out_scale = out_scale;
    a.D = s.head_dim;
    a.key_pages = static_cast<const uint16_t*>(key_pages);
    a.value_pages = static_cast<const uint16_t*>(value_pages);
    a.window = window;
    a.sinks = sinks;
    const int grid = workspace ? window_split_grid(s, page_size, max_context_len, window, sinks, dev) : 0;
    if (grid > 0 && workspace_bytes >= prefill_split_workspace_bytes(grid) &&
        (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0) {
        const cudaError_t e = run_split(qmap, kmap, vmap, a, dev, grid, workspace, stream);
        if (e != cudaErrorNotSupported)
            return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    const cudaError_t e = launch_prefill_pairs(qmap, kmap, vmap, omap, a, dev->id, dev->sm_count,
                                               nullptr, 0, stream);
    return e == cudaSuccess ? PA_OK : e == cudaErrorNotSupported ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
}

// (request, KV head, 16-row tile) count of a call: the limit kMaxSegments
// applies to it.
int64_t decode_segments(const pa_shape& s)
{
    const int64_t G = s.num_q_heads / s.num_kv_heads;
    const int64_t MT = (G * s.q_len + kDecodeRows - 1) / kDecodeRows;
    return int64_t(s.batch) * s.num_kv_heads * MT;
}

}  // namespace

DecodePlan decode_plan(const pa_shape& s, bool fp8)
{
    DecodePlan p;
    const int64_t G = s.num_q_heads / s.num_kv_heads;
    p.MT = int32_t((G * s.q_len + kDecodeRows - 1) / kDecodeRows);
    p.TG = fp8 || p.MT <= 1 ? 1 : p.MT == 2 ? 2 : 4;
    p.MS = (p.MT + p.TG - 1) / p.TG;
    p.nseg = int64_t(s.batch) * s.num_kv_heads * p.MS;
    return p;
}

namespace {

// What a split-KV call does beyond full attention.
struct DecodeExtra {
    DecodeMode mode = kFull;
    int32_t window = 0, sinks = 0;   // kWindow
    float* scores = nullptr;         // kScores
    float2* row_state = nullptr;
    int64_t score_stride = 0;
    int32_t score_cap = 0;
};

// Runs the split-KV kernel. whole_segments = 1 gives every block whole
// segments (no partial states, no workspace).
pa_status run_split_kv(const void* query, const void* key_pages, const void* value_pages,
                       const int32_t* block_table, const int32_t* context_lens,
                       int32_t page_size, float scale, int causal, void* out,
                       const pa_shape& s, int32_t max_context_len, void* workspace,
                       size_t workspace_bytes, int whole_segments, cudaStream_t stream,
                       int dense = 0, int fp8 = 0, float k_scale = 1.f, float v_scale = 1.f,
                       const DecodeExtra& extra = DecodeExtra())
{
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    const int G = s.num_q_heads / s.num_kv_heads;
    const int64_t R = int64_t(G) * s.q_len;
    if (R >= (int64_t(1) << 30) || decode_segments(s) > kMaxSegments)
        return PA_ERR_UNSUPPORTED;
    const DecodePlan plan = decode_plan(s, fp8 != 0);
    const int64_t nseg = plan.nseg;
    const size_t smem = decode_smem_bytes(s.head_dim, s.batch, fp8 != 0, plan.TG) +
                        decode_static_smem_bytes(fp8 != 0);
    if (smem > size_t(dev->max_smem_optin))
        return PA_ERR_UNSUPPORTED;  // batch too large for the per-block prefix table

    const int grid_max = decode_max_grid(dev->sm_count);
    int64_t grid = grid_max;
    int64_t granules = 0;                  // of 64 keys, at most
    if (whole_segments) {
        grid = nseg < grid_max ? nseg : grid_max;
    } else if (max_context_len > 0) {
        int64_t gran = (int64_t(max_context_len) + kDecodeTokens - 1) / kDecodeTokens;
        if (extra.mode == kWindow) {
            // a sliding window's two runs of keys, the second from a page border
            const int64_t runs =
                (int64_t(extra.sinks) + kDecodeTokens - 1) / kDecodeTokens +
                (int64_t(extra.window) + s.q_len + 2 * kDecodeTokens - 3) / kDecodeTokens;
            gran = std::min(gran, runs);
        }
        granules = nseg * (gran > 0 ? gran : 1);
        if (granules < grid)
            grid = granules;
    }
    if (grid < 1)
        grid = 1;

    const bool rows = extra.mode != kFull && !whole_segments &&
                      decode_rows_takes(s, dev->max_smem_optin);
    DecodeArgs a;
    memset(&a, 0, sizeof a);
    if (rows) {
        if (!workspace ||
            workspace_bytes < decode_rows_workspace_bytes(s, fp8 ? kE4m3Pool : kBf16Pool, extra.mode, dev->sm_count) ||
            (reinterpret_cast<uintptr_t>(workspace) & 15u))
            return PA_ERR_WORKSPACE;
    } else if (!whole_segments) {
        const size_t need = decode_workspace_bytes(nseg, grid_max, s.head_dim, plan.TG);
        if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u))
            return PA_ERR_WORKSPACE;
        a.partials = static_cast<float*>(workspace);
    }
    a.q = static_cast<const uint16_t*>(query);
    a.out = static_cast<uint16_t*>(out);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.L = s.q_len;
    a.D = s.head_dim;
    a.ps = page_size;
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.G = G;
    a.R = int32_t(R);
    a.MS = plan.MS;
    a.TG = plan.TG;
    a.box_rows = page_size < kDecodeTokens ? page_size : kDecodeTokens;
    a.swz = a.box_rows >= 8 ? 7 : 0;
    a.whole_segments = whole_segments;
    a.dense = dense;
    // e4m3 pages: the kernel's K and V fragments hold the code values; the
    // per-tensor scales go into the softmax scale and the output
    a.scale_log2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.f);
    a.causal = causal ? 1 : 0;
    a.fp8 = fp8 ? 1 : 0;
    a.v_scale = fp8 ? v_scale : 1.f;
    a.mode = extra.mode;
    a.window = extra.window;
    a.sinks = extra.sinks;
    a.scores = extra.scores;
    a.row_state = extra.row_state;
    a.score_stride = extra.score_stride;
    a.score_cap = extra.score_cap;
    if (rows) {
        CUtensorMap kmap, vmap;
        const int kind = fp8 ? kE4m3Pool : kBf16Pool;
        a.box_rows = decode_rows_box(s, kind, page_size);
        a.swz = a.box_rows >= 8 ? 7 : 0;
        if ((st = encode_pool_map(&kmap, key_pages, s, page_size, fp8 != 0, a.box_rows)) != PA_OK ||
            (st = encode_pool_map(&vmap, value_pages, s, page_size, fp8 != 0, a.box_rows)) != PA_OK)
            return st;
        while ((1 << a.ps_shift) < page_size)
            ++a.ps_shift;
        const int rows_grid =
            decode_rows_launch_grid(s, kind, extra.mode, max_context_len > 0 ? granules : 0, dev->sm_count);
        return launch_decode_rows(kmap, vmap, a, s, kind, rows_grid, workspace, dev->id, stream) == cudaSuccess
                   ? PA_OK
                   : PA_ERR_CUDA;
    }
    a.debug_unset_wait = t_arm_unset_wait ? 1 : 0;
    t_arm_unset_wait = false;
    CUtensorMap kmap, vmap;
    if ((st = encode_pool_map(&kmap, key_pages, s, page_size, fp8 != 0)) != PA_OK)
        return st;
    if ((st = encode_pool_map(&vmap, value_pages, s, page_size, fp8 != 0)) != PA_OK)
        return st;
    CUtensorMap qmap;
    const uint64_t q_rows = uint64_t(s.batch) * s.num_q_heads * s.q_len;
    if ((st = encode_rows_map(&qmap, query, q_rows, uint32_t(kDecodeRows), uint32_t(s.head_dim))) !=
        PA_OK)
        return st;
    return launch_decode(kmap, vmap, qmap, a, int(grid), dev->id, stream) == cudaSuccess ? PA_OK
                                                                                   : PA_ERR_CUDA;
}

}  // namespace

pa_status validate_decode(const void* query, const void* key_pages, const void* value_pages,
                          const int32_t* block_table, const int32_t* context_lens,
                          int32_t page_size, float scale, const void* out, const pa_shape& s)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, s);
    if (st != PA_OK)
        return st;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    const int64_t R = int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len;
    if (R >= (int64_t(1) << 30) || decode_segments(s) > kMaxSegments)
        return PA_ERR_UNSUPPORTED;
    const size_t smem = std::max(decode_smem_bytes(s.head_dim, s.batch),
                                 decode_smem_bytes(s.head_dim, s.batch, false,
                                                   decode_plan(s, false).TG));
    if (smem > size_t(dev->max_smem_optin))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

int64_t decode_segment_count(const pa_shape& s) { return decode_segments(s); }

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_append_kv(const void* key, const void* value, void* key_pages, void* value_pages,
                       const int32_t* slot_mapping, int32_t page_size, pa_shape shape,
                       void* stream)
{
    if (!key || !value || !key_pages || !value_pages || !slot_mapping)
        return PA_ERR_INVALID_ARG;
    if (shape.batch <= 0 || shape.num_kv_heads <= 0 || shape.q_len < 0 || shape.num_pages <= 0 ||
        shape.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_pages) || !aligned16(value_pages))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 64 && shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    if (!pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (2 * int64_t(shape.batch) * shape.q_len * shape.num_kv_heads * (shape.head_dim / 8) >=
        (int64_t(1) << 40))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (shape.q_len == 0)
        return PA_OK;
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.key = static_cast<const uint16_t*>(key);
    a.value = static_cast<const uint16_t*>(value);
    a.key_pages = static_cast<uint16_t*>(key_pages);
    a.value_pages = static_cast<uint16_t*>(value_pages);
    a.slot_mapping = slot_mapping;
    a.err = dev->err;
    a.B = shape.batch;
    a.L_new = shape.q_len;
    a.H_kv = shape.num_kv_heads;
    a.D = shape.head_dim;
    a.ps = page_size;
    a.num_pages = shape.num_pages;
    return launch_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                               : PA_ERR_CUDA;
}

size_t pa_decode_workspace_bytes(pa_shape shape)
{
    if (shape.batch <= 0 || shape.num_q_heads <= 0 || shape.num_kv_heads <= 0 ||
        shape.q_len <= 0 || shape.num_q_heads % shape.num_kv_heads != 0 ||
        (shape.head_dim != 64 && shape.head_dim != 128) ||
        decode_segments(shape) > kMaxSegments)
        return 0;
    DeviceInfo* dev;
    if (device_info(&dev) != PA_OK)
        return 0;
    // The bf16 plan's need; an e4m3 call's (one row tile per segment) is
    // never larger.
    const DecodePlan plan = decode_plan(shape, false);
    return decode_workspace_bytes(plan.nseg, decode_max_grid(dev->sm_count), shape.head_dim,
                                  plan.TG);
}

namespace {

// Prefill over e4m3 pools: the workspace holds the bf16 copies of K and V
// (B * P2 pages of [H_kv, 128, 128]), the copies' page table, then (256-byte
// aligned) the split prefill's workspace where that kernel serves the shape.
struct Fp8PrefillPlan {
    int64_t P2 = 0;
    pa_shape copy{};
    size_t kv_bytes = 0, table_off = 0, split_off = 0, split_bytes = 0, piece_bytes = 0, total = 0;
};

pa_status plan_prefill_fp8(const pa_shape& s, int32_t max_context_len, DeviceInfo* dev,
                           Fp8PrefillPlan* p)
{
    if (max_context_len < 0 || s.batch <= 0 || s.num_kv_heads <= 0 || s.num_q_heads <= 0 || s.q_len <= 0)
        return PA_ERR_INVALID_ARG;
    if (s.num_q_heads % s.num_kv_heads != 0)
        return PA_ERR_UNSUPPORTED;
    p->P2 = fp8_copy_pages(max_context_len);
    const int64_t pages = int64_t(s.batch) * p->P2;
    if (pages * s.num_kv_heads * 128 >= (int64_t(1) << 31) || p->P2 * 128 >= (int64_t(1) << 30))
        return PA_ERR_UNSUPPORTED;
    p->copy = s;
    p->copy.head_dim = 128;
    p->copy.num_pages = int32_t(pages);
    p->copy.max_pages = int32_t(p->P2);
    p->kv_bytes = size_t(pages) * s.num_kv_heads * 128 * 128 * 2;
    p->table_off = 2 * p->kv_bytes;
    const size_t table_bytes = size_t(pages) * 4;
    p->split_off = (p->table_off + table_bytes + 255) & ~size_t(255);
    // the kernel choice of pa_attention's prefill route (split below 1.5
    // items per SM; from there to 2 items per SM the pairs kernel's tail
    // pieces, in the same place)
    const int64_t items = prefill_pair_items(s);
    const bool few = 2 * items < 3 * int64_t(dev->sm_count);
    p->split_bytes = few ? split_prefill_need(p->copy, 128, dev) : 0;
    p->piece_bytes = !few && items <= 2 * int64_t(dev->sm_count) && split_prefill_need(p->copy, 128, dev) > 0
                         ? prefill_pairs_workspace_bytes(dev->sm_count)
                         : 0;
    p->total = p->split_off + (p->split_bytes > p->piece_bytes ? p->split_bytes : p->piece_bytes);
    return PA_OK;
}

}  // namespace

size_t pa_prefill_fp8_workspace_bytes(pa_shape shape, int32_t max_context_len)
{
    if (shape.head_dim != 128)
        return 0;
    DeviceInfo* dev;
    if (device_info(&dev) != PA_OK)
        return 0;
    Fp8PrefillPlan p;
    if (plan_prefill_fp8(shape, max_context_len, dev, &p) != PA_OK)
        return 0;
    return p.total;
}

pa_status pa_prefill_fp8(const void* query, const void* key_pages, const void* value_pages,
                         const int32_t* block_table, const int32_t* context_lens,
                         int32_t page_size, float scale, float k_scale, float v_scale, int causal,
                         void* out, pa_shape shape, int32_t max_context_len, void* workspace,
                         size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (!(k_scale > 0.f) || !isfinite(k_scale) || !(v_scale > 0.f) || !isfinite(v_scale))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    Fp8PrefillPlan p;
    if ((st = plan_prefill_fp8(shape, max_context_len, dev, &p)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < p.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    Fp8PagesArgs c;
    memset(&c, 0, sizeof c);
    c.key_pages = static_cast<const uint8_t*>(key_pages);
    c.value_pages = static_cast<const uint8_t*>(value_pages);
    c.block_table = block_table;
    c.context_lens = context_lens;
    c.key_out = reinterpret_cast<uint16_t*>(w);
    c.value_out = reinterpret_cast<uint16_t*>(w + p.kv_bytes);
    c.table_out = reinterpret_cast<int32_t*>(w + p.table_off);
    c.err = dev->err;
    c.B = shape.batch;
    c.H_kv = shape.num_kv_heads;
    c.ps = page_size;
    c.max_pages = shape.max_pages;
    c.num_pages = shape.num_pages;
    c.P2 = int32_t(p.P2);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_fp8_pages_to_bf16(c, s) != cudaSuccess)
        return PA_ERR_CUDA;
    // k_scale into the softmax scale, v_scale into the output normalisation
    return run_prefill_tc(query, c.key_out, c.value_out, c.table_out, context_lens, 128,
                          scale * k_scale, causal, out, p.copy, s,
                          p.split_bytes ? w + p.split_off : nullptr, p.split_bytes, v_scale,
                          p.piece_bytes ? w + p.split_off : nullptr, p.piece_bytes);
}

namespace {

// Route of pa_attention_fp8: the e4m3 decode kernel carries one 16-row tile
// per segment (its K/V are read once per tile), so it takes query chunks of
// at most 8 rows per request, the rule of Week 3 Day 4, "Task 2".
int32_t route_fp8(const pa_shape& shape)
{
    if (shape.q_len <= 0)
        return -1;
    return shape.q_len <= 8 ? 0 : 1;
}

}  // namespace

size_t pa_attention_fp8_workspace_bytes(pa_shape shape, int32_t max_context_len)
{
    const int32_t route = route_fp8(shape);
    if (route < 0 || shape.head_dim != 128)
        return 0;
    return route == 0 ? pa_decode_workspace_bytes(shape)
                      : pa_prefill_fp8_workspace_bytes(shape, max_context_len);
}

pa_status pa_attention_fp8(const void* query, const void* key_pages, const void* value_pages,
                           const int32_t* block_table, const int32_t* context_lens,
                           int32_t page_size, float scale, float k_scale, float v_scale,
                           int causal, void* out, pa_shape shape, int32_t max_context_len,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    const int32_t route = route_fp8(shape);
    if (route < 0)
        return PA_ERR_INVALID_ARG;
    if (route == 0)
        return pa_decode_fp8(query, key_pages, value_pages, block_table, context_lens, page_size,
                             scale, k_scale, v_scale, causal, out, shape, max_context_len,
                             workspace, workspace_bytes, stream);
    return pa_prefill_fp8(query, key_pages, value_pages, block_table, context_lens, page_size,
                          scale, k_scale, v_scale, causal, out, shape, max_context_len, workspace,
                          workspace_bytes, stream);
}

pa_status pa_append_kv_fp8(const void* key, const void* value, void* key_pages,
                           void* value_pages, const int32_t* slot_mapping, int32_t page_size,
                           float k_scale, float v_scale, pa_shape shape, void* stream)
{
    if (!key || !value || !key_pages || !value_pages || !slot_mapping)
        return PA_ERR_INVALID_ARG;
    if (shape.batch <= 0 || shape.num_kv_heads <= 0 || shape.q_len < 0 || shape.num_pages <= 0 ||
        shape.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!(k_scale > 0.f) || !isfinite(k_scale) || !(v_scale > 0.f) || !isfinite(v_scale))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_pages) || !aligned16(value_pages))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    if (!pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (2 * int64_t(shape.batch) * shape.q_len * shape.num_kv_heads * (shape.head_dim / 8) >=
        (int64_t(1) << 40))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (shape.q_len == 0)
        return PA_OK;
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.key = static_cast<const uint16_t*>(key);
    a.value = static_cast<const uint16_t*>(value);
    a.key_pages = static_cast<uint16_t*>(key_pages);     // byte pages; the kernel casts back
    a.value_pages = static_cast<uint16_t*>(value_pages);
    a.slot_mapping = slot_mapping;
    a.err = dev->err;
    a.B = shape.batch;
    a.L_new = shape.q_len;
    a.H_kv = shape.num_kv_heads;
    a.D = shape.head_dim;
    a.ps = page_size;
    a.num_pages = shape.num_pages;
    a.fp8 = 1;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return launch_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                               : PA_ERR_CUDA;
}

namespace {

bool ranges_overlap(const void* p, uint64_t p_bytes, const void* q, uint64_t q_bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + q_bytes && b < a + p_bytes;
}

// Both pools' forms: fp8 with their scales, or bf16 (scales 1).
pa_status run_norm_rope_append(const void* qkv, int64_t batch_stride, int64_t token_stride,
                               const void* q_weight, const void* k_weight, float eps,
                               const float* cos_sin, int32_t rotary_dim, int32_t table_len,
                               int interleaved, const int32_t* positions, void* query,
                               void* key_pages, void* value_pages, const int32_t* slot_mapping,
                               int32_t page_size, int fp8, float k_scale, float v_scale,
                               const pa_shape& s, void* stream)
{
    if (!qkv || !query || !key_pages || !value_pages || !slot_mapping)
        return PA_ERR_INVALID_ARG;
    if (s.batch <= 0 || s.num_q_heads <= 0 || s.num_kv_heads <= 0 || s.q_len < 0 ||
        s.num_pages <= 0 || s.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(query) || !aligned16(key_pages) || !aligned16(value_pages) ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin))
        return PA_ERR_INVALID_ARG;
    if ((q_weight || k_weight) && (!(eps >= 0.f) || !isfinite(eps)))
        return PA_ERR_INVALID_ARG;
    if (fp8 && (!(k_scale > 0.f) || !isfinite(k_scale) || !(v_scale > 0.f) || !isfinite(v_scale)))
        return PA_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim > s.head_dim ||
        (rotary_dim > 0 && (!cos_sin || !positions || table_len <= 0)))
        return PA_ERR_INVALID_ARG;
    if ((s.head_dim != 64 && s.head_dim != 128) || (fp8 && s.head_dim != 128) ||
        rotary_dim % 16 != 0)
        return PA_ERR_UNSUPPORTED;
    if (s.num_q_heads % s.num_kv_heads != 0 || !pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    const int64_t heads = int64_t(s.num_q_heads) + 2 * int64_t(s.num_kv_heads);
    if (heads >= (1 << 20) || int64_t(s.batch) * s.q_len * heads >= (int64_t(1) << 34))
        return PA_ERR_UNSUPPORTED;
    const int64_t row = heads * s.head_dim;
    if (token_stride % 8 != 0 || batch_stride % 8 != 0 || token_stride < 0 || batch_stride < 0 ||
        (s.q_len > 1 && token_stride < row) || (s.batch > 1 && batch_stride < row))
        return PA_ERR_INVALID_ARG;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (s.q_len == 0)
        return PA_OK;
    // The rows are read by other threads than those that write the queries.
    const uint64_t in_bytes =
        2 * uint64_t((s.batch - 1) * batch_stride + (s.q_len - 1) * token_stride + row);
    const uint64_t q_bytes = 2 * uint64_t(s.batch) * s.num_q_heads * s.q_len * s.head_dim;
    if (ranges_overlap(qkv, in_bytes, query, q_bytes))
        return PA_ERR_INVALID_ARG;
    NormRopeArgs a;
    memset(&a, 0, sizeof a);
    a.qkv = static_cast<const uint16_t*>(qkv);
    a.batch_stride = batch_stride;
    a.token_stride = token_stride;
    a.q_weight = static_cast<const uint16_t*>(q_weight);
    a.k_weight = static_cast<const uint16_t*>(k_weight);
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.query = static_cast<uint16_t*>(query);
    a.key_pages = static_cast<uint16_t*>(key_pages);
    a.value_pages = static_cast<uint16_t*>(value_pages);
    a.slot_mapping = slot_mapping;
    a.err = dev->err;
    a.B = s.batch;
    a.L = s.q_len;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.D = s.head_dim;
    while ((1 << a.ps_shift) < page_size)
        ++a.ps_shift;
    a.num_pages = s.num_pages;
    a.rotary_dim = rotary_dim;
    a.table_len = table_len;
    a.interleaved = interleaved ? 1 : 0;
    a.fp8 = fp8;
    a.eps = eps;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return launch_norm_rope_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

pa_status pa_qk_norm_rope_append(const void* qkv, int64_t qkv_batch_stride,
                                 int64_t qkv_token_stride, const void* q_weight,
                                 const void* k_weight, float eps, const float* cos_sin,
                                 int32_t rotary_dim, int32_t table_len, int interleaved,
                                 const int32_t* positions, void* query, void* key_pages,
                                 void* value_pages, const int32_t* slot_mapping,
                                 int32_t page_size, pa_shape shape, void* stream)
{
    return run_norm_rope_append(qkv, qkv_batch_stride, qkv_token_stride, q_weight, k_weight, eps,
                                cos_sin, rotary_dim, table_len, interleaved, positions, query,
                                key_pages, value_pages, slot_mapping, page_size, 0, 1.f, 1.f,
                                shape, stream);
}

pa_status pa_qk_norm_rope_append_fp8(const void* qkv, int64_t qkv_batch_stride,
                                     int64_t qkv_token_stride, const void* q_weight,
                                     const void* k_weight, float eps, const float* cos_sin,
                                     int32_t rotary_dim, int32_t table_len, int interleaved,
                                     const int32_t* positions, void* query, void* key_pages,
                                     void* value_pages, const int32_t* slot_mapping,
                                     int32_t page_size, float k_scale, float v_scale,
                                     pa_shape shape, void* stream)
{
    return run_norm_rope_append(qkv, qkv_batch_stride, qkv_token_stride, q_weight, k_weight, eps,
                                cos_sin, rotary_dim, table_len, interleaved, positions, query,
                                key_pages, value_pages, slot_mapping, page_size, 1, k_scale,
                                v_scale, shape, stream);
}

namespace {

pa_status run_evict(void* key_pages, void* value_pages, float* weight_pages,
                    const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                    int32_t keep, int32_t sinks, int32_t recent, const int32_t* dst_block_table,
                    int32_t dst_max_pages, int32_t* kept, int32_t* new_lens, int fp8,
                    const pa_shape& s, void* stream)
{
    if (!key_pages || !value_pages || !weight_pages || !block_table || !context_lens ||
        !dst_block_table || !kept || !new_lens)
        return PA_ERR_INVALID_ARG;
    if (s.batch <= 0 || s.num_kv_heads <= 0 || s.num_pages <= 0 || s.max_pages <= 0 ||
        s.head_dim <= 0 || dst_max_pages <= 0)
        return PA_ERR_INVALID_ARG;
    if (keep <= 0 || sinks < 0 || recent < 0 || int64_t(sinks) + recent > keep)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key_pages) || !aligned16(value_pages) ||
        (reinterpret_cast<uintptr_t>(weight_pages) & 3u) != 0)
        return PA_ERR_INVALID_ARG;
    if ((s.head_dim != 64 && s.head_dim != 128) || (fp8 && s.head_dim != 128) ||
        !pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(s.num_pages) * s.num_kv_heads * page_size >= (int64_t(1) << 31) ||
        int64_t(s.max_pages) * page_size >= (int64_t(1) << 30) ||
        int64_t(dst_max_pages) * page_size >= (int64_t(1) << 30) || keep >= (1 << 30) ||
        int64_t(s.batch) * s.num_kv_heads >= (int64_t(1) << 24))
        return PA_ERR_UNSUPPORTED;
    // Every kept row needs a place.
    const int64_t most = std::min(int64_t(keep), int64_t(s.max_pages) * page_size);
    if (int64_t(dst_max_pages) * page_size < most)
        return PA_ERR_INVALID_ARG;
    // In place the two tables are one: rows of another width would be other requests'.
    if (dst_block_table == block_table && s.batch > 1 && dst_max_pages != s.max_pages)
        return PA_ERR_INVALID_ARG;
    // The kernels read the lengths and the table after new_lens and kept are written.
    const uint64_t heads = uint64_t(s.batch) * s.num_kv_heads;
    const uint64_t kept_bytes = heads * keep * 4, len_bytes = uint64_t(s.batch) * 4;
    for (const void* out : {static_cast<const void*>(kept), static_cast<const void*>(new_lens)}) {
        const uint64_t bytes = out == kept ? kept_bytes : len_bytes;
        if (ranges_overlap(out, bytes, context_lens, len_bytes) ||
            ranges_overlap(out, bytes, block_table, uint64_t(s.batch) * s.max_pages * 4) ||
            ranges_overlap(out, bytes, dst_block_table, uint64_t(s.batch) * dst_max_pages * 4))
            return PA_ERR_INVALID_ARG;
    }
    if (ranges_overlap(kept, kept_bytes, new_lens, len_bytes))
        return PA_ERR_INVALID_ARG;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    EvictArgs a;
    memset(&a, 0, sizeof a);
    a.key_pages = key_pages;
    a.value_pages = value_pages;
    a.weight_pages = weight_pages;
    a.block_table = block_table;
    a.dst_table = dst_block_table;
    a.context_lens = context_lens;
    a.kept = kept;
    a.new_lens = new_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_kv = s.num_kv_heads;
    a.row_bytes = s.head_dim * (fp8 ? 1 : 2);
    while ((1 << a.ps_shift) < page_size)
        ++a.ps_shift;
    a.num_pages = s.num_pages;
    a.max_pages = s.max_pages;
    a.dst_max_pages = dst_max_pages;
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    return launch_evict(a, dev->id, dev->sm_count, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

pa_status pa_kv_evict(void* key_pages, void* value_pages, float* weight_pages,
                      const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                      int32_t keep, int32_t sinks, int32_t recent, const int32_t* dst_block_table,
                      int32_t dst_max_pages, int32_t* kept, int32_t* new_lens, pa_shape shape,
                      void* stream)
{
    return run_evict(key_pages, value_pages, weight_pages, block_table, context_lens, page_size,
                     keep, sinks, recent, dst_block_table, dst_max_pages, kept, new_lens, 0, shape,
                     stream);
}

pa_status pa_kv_evict_fp8(void* key_pages, void* value_pages, float* weight_pages,
                          const int32_t* block_table, const int32_t* context_lens,
                          int32_t page_size, int32_t keep, int32_t sinks, int32_t recent,
                          const int32_t* dst_block_table, int32_t dst_max_pages, int32_t* kept,
                          int32_t* new_lens, pa_shape shape, void* stream)
{
    return run_evict(key_pages, value_pages, weight_pages, block_table, context_lens, page_size,
                     keep, sinks, recent, dst_block_table, dst_max_pages, kept, new_lens, 1, shape,
                     stream);
}

pa_status pa_decode_fp8(const void* query, const void* key_pages, const void* value_pages,
                        const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                        float scale, float k_scale, float v_scale, int causal, void* out,
                        pa_shape shape, int32_t max_context_len, void* workspace,
                        size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (!(k_scale > 0.f) || !isfinite(k_scale) || !(v_scale > 0.f) || !isfinite(v_scale))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    return run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                        causal, out, shape, max_context_len, workspace, workspace_bytes, 0,
                        static_cast<cudaStream_t>(stream), 0, 1, k_scale, v_scale);
}

pa_status pa_decode(const void* query, const void* key_pages, const void* value_pages,
                    const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                    float scale, int causal, void* out, pa_shape shape, int32_t max_context_len,
                    void* workspace, size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    return run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size,
                        scale, causal, out, shape, max_context_len, workspace, workspace_bytes,
                        0, static_cast<cudaStream_t>(stream));
}

namespace {

bool bad_scales(float k_scale, float v_scale)
{
    return !(k_scale > 0.f) || !isfinite(k_scale) || !(v_scale > 0.f) || !isfinite(v_scale);
}

// Checks of a sliding window, and the window cut to what positions can reach.
pa_status check_window(int32_t window, int32_t sinks, int32_t* cut)
{
    if (window <= 0 || sinks < 0)
        return PA_ERR_INVALID_ARG;
    *cut = std::min(window, 1 << 30);
    return PA_OK;
}

pa_status run_decode_window(const void* query, const void* key_pages, const void* value_pages,
                            const int32_t* block_table, const int32_t* context_lens,
                            int32_t page_size, float scale, int fp8, float k_scale, float v_scale,
                            int32_t window, int32_t sinks, void* out, const pa_shape& shape,
                            int32_t max_context_len, void* workspace, size_t workspace_bytes,
                            void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    DecodeExtra extra;
    extra.mode = kWindow;
    if ((st = check_window(window, sinks, &extra.window)) != PA_OK)
        return st;
    extra.sinks = std::min(sinks, 1 << 30);
    if (fp8 && bad_scales(k_scale, v_scale))
        return PA_ERR_INVALID_ARG;
    if (fp8 && shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    return run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                        1, out, shape, max_context_len, workspace, workspace_bytes, 0,
                        static_cast<cudaStream_t>(stream), 0, fp8, k_scale, v_scale, extra);
}

// Prefill over e4m3 pools with a sliding window: the tokens that some row sees
// as bf16 copies (P1 pages of 128 tokens a request), and their table of P2
// entries a request.
struct WindowCopyPlan {
    int64_t P1 = 0, P2 = 0;
    pa_shape copy{};
    size_t kv_bytes = 0, table_off = 0, split_off = 0, split_bytes = 0, total = 0;
};

pa_status plan_window_copy(const pa_shape& s, int32_t max_context_len, int32_t window,
                           int32_t sinks, WindowCopyPlan* p)
{
    if (max_context_len < 0 || s.batch <= 0 || s.num_kv_heads <= 0 || s.num_q_heads <= 0 ||
        s.q_len <= 0)
        return PA_ERR_INVALID_ARG;
    p->P2 = fp8_copy_pages(max_context_len);
    p->P1 = fp8_window_pages(max_context_len, window, sinks, s.q_len);
    const int64_t pages = int64_t(s.batch) * p->P1;
    if (pages * s.num_kv_heads * 128 >= (int64_t(1) << 31) || p->P2 * 128 >= (int64_t(1) << 30) ||
        int64_t(s.batch) * p->P2 >= (int64_t(1) << 31))
        return PA_ERR_UNSUPPORTED;
    p->copy = s;
    p->copy.num_pages = int32_t(pages);
    p->copy.max_pages = int32_t(p->P2);
    p->kv_bytes = size_t(pages) * s.num_kv_heads * 128 * 128 * 2;
    p->table_off = 2 * p->kv_bytes;
    p->split_off = (p->table_off + size_t(s.batch) * size_t(p->P2) * 4 + 255) & ~size_t(255);
    DeviceInfo* dev;
    const pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    p->split_bytes = window_split_need(s, 128, max_context_len, window, sinks, dev);
    p->total = p->split_off + p->split_bytes;
    return PA_OK;
}

// Keys that a row of the call can see at most: the context that matters to the
// choice of the kernel.
int32_t window_reach(const pa_shape& s, int32_t max_context_len, int32_t window, int32_t sinks)
{
    const int64_t reach = int64_t(window) + sinks + s.q_len;
    return max_context_len > 0 && max_context_len < reach ? max_context_len
                                                          : int32_t(std::min<int64_t>(reach, 1 << 30));
}

// Workspace of a weight-accumulating decode: the decode's, then the scores of
// every row (score_stride columns), then the row states.
struct WeightPlan {
    size_t score_off = 0, state_off = 0, total = 0;
    int64_t stride = 0;
};

pa_status plan_weights(const pa_shape& s, int32_t max_context_len, WeightPlan* p)
{
    if (max_context_len <= 0)
        return PA_ERR_INVALID_ARG;
    const size_t decode = pa_decode_window_workspace_bytes(s);   // the same kernels
    if (decode == 0)
        return PA_ERR_UNSUPPORTED;
    p->stride = (int64_t(max_context_len) + 63) / 64 * 64;
    const int64_t rows = int64_t(s.batch) * s.num_q_heads * s.q_len;
    if (max_context_len > (1 << 30) || rows >= (int64_t(1) << 31) ||
        rows * p->stride >= (int64_t(1) << 38))
        return PA_ERR_UNSUPPORTED;
    p->score_off = (decode + 255) & ~size_t(255);
    p->state_off = p->score_off + size_t(rows) * size_t(p->stride) * sizeof(float);
    p->total = p->state_off + size_t(rows) * sizeof(float2);
    return PA_OK;
}

pa_status run_decode_weights(const void* query, const void* key_pages, const void* value_pages,
                             float* weight_pages, const int32_t* block_table,
                             const int32_t* context_lens, int32_t page_size, float scale, int fp8,
                             float k_scale, float v_scale, int causal, float decay, void* out,
                             const pa_shape& shape, int32_t max_context_len, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (!weight_pages || (reinterpret_cast<uintptr_t>(weight_pages) & 3u) != 0 ||
        !(decay >= 0.f) || !isfinite(decay) || max_context_len <= 0)
        return PA_ERR_INVALID_ARG;
    if (fp8 && bad_scales(k_scale, v_scale))
        return PA_ERR_INVALID_ARG;
    if (fp8 && shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    WeightPlan p;
    if ((st = plan_weights(shape, max_context_len, &p)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < p.total || (reinterpret_cast<uintptr_t>(workspace) & 15u))
        return PA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    DecodeExtra extra;
    extra.mode = kScores;
    extra.scores = reinterpret_cast<float*>(w + p.score_off);
    extra.row_state = reinterpret_cast<float2*>(w + p.state_off);
    extra.score_stride = p.stride;
    extra.score_cap = max_context_len;
    WeightArgs a;
    memset(&a, 0, sizeof a);
    a.scores = extra.scores;
    a.row_state = extra.row_state;
    a.weight_pages = weight_pages;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.score_stride = p.stride;
    a.B = shape.batch;
    a.H_kv = shape.num_kv_heads;
    a.R = int32_t(int64_t(shape.num_q_heads / shape.num_kv_heads) * shape.q_len);
    a.L = shape.q_len;
    while ((1 << a.ps_shift) < page_size)
        ++a.ps_shift;
    a.max_pages = shape.max_pages;
    a.num_pages = shape.num_pages;
    a.score_cap = max_context_len;
    a.decay = decay;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                      causal, out, shape, max_context_len, workspace, p.score_off, 0, s, 0, fp8,
                      k_scale, v_scale, extra);
    if (st != PA_OK)
        return st;
    return launch_accumulate_weights(a, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

size_t pa_decode_window_workspace_bytes(pa_shape shape)
{
    const size_t many = pa_decode_workspace_bytes(shape);
    DeviceInfo* dev;
    if (many == 0 || device_info(&dev) != PA_OK)
        return 0;
    return decode_rows_takes(shape, dev->max_smem_optin)
               ? decode_rows_workspace_bytes(shape, kBf16Pool, kWindow, dev->sm_count)
               : many;
}

pa_status pa_decode_window(const void* query, const void* key_pages, const void* value_pages,
                           const int32_t* block_table, const int32_t* context_lens,
                           int32_t page_size, float scale, int32_t window, int32_t sinks, void* out,
                           pa_shape shape, int32_t max_context_len, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    return run_decode_window(query, key_pages, value_pages, block_table, context_lens, page_size,
                             scale, 0, 1.f, 1.f, window, sinks, out, shape, max_context_len,
                             workspace, workspace_bytes, stream);
}

pa_status pa_decode_window_fp8(const void* query, const void* key_pages, const void* value_pages,
                               const int32_t* block_table, const int32_t* context_lens,
                               int32_t page_size, float scale, float k_scale, float v_scale,
                               int32_t window, int32_t sinks, void* out, pa_shape shape,
                               int32_t max_context_len, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    return run_decode_window(query, key_pages, value_pages, block_table, context_lens, page_size,
                             scale, 1, k_scale, v_scale, window, sinks, out, shape,
                             max_context_len, workspace, workspace_bytes, stream);
}

namespace {

pa_status run_window_prefill(const void* query, const void* key_pages, const void* value_pages,
                             const int32_t* block_table, const int32_t* context_lens,
                             int32_t page_size, float scale, int32_t window, int32_t sinks,
                             void* out, const pa_shape& shape, int32_t max_context_len,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    DecodeExtra extra;
    extra.mode = kWindow;
    if ((st = check_window(window, sinks, &extra.window)) != PA_OK)
        return st;
    extra.sinks = std::min(sinks, 1 << 30);
    st = run_prefill_window(query, key_pages, value_pages, block_table, context_lens, page_size,
                            scale, extra.window, extra.sinks, 1.f, out, shape, max_context_len,
                            workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    if (st != PA_ERR_UNSUPPORTED)
        return st;
    // Without the pairs kernel's register split: the split-KV kernel with
    // whole segments per block, as pa_prefill.
    return run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                        1, out, shape, 0, nullptr, 0, 1, static_cast<cudaStream_t>(stream), 0, 0,
                        1.f, 1.f, extra);
}

}  // namespace

pa_status pa_prefill_window(const void* query, const void* key_pages, const void* value_pages,
                            const int32_t* block_table, const int32_t* context_lens,
                            int32_t page_size, float scale, int32_t window, int32_t sinks,
                            void* out, pa_shape shape, void* stream)
{
    return run_window_prefill(query, key_pages, value_pages, block_table, context_lens, page_size,
                              scale, window, sinks, out, shape, 0, nullptr, 0, stream);
}

size_t pa_attention_window_workspace_bytes(pa_shape shape, int32_t page_size,
                                           int32_t max_context_len, int32_t window, int32_t sinks)
{
    if (!pow2_in(page_size, 1, 256) || window <= 0 || sinks < 0 || max_context_len < 0)
        return 0;
    const int32_t route =
        pa_attention_route(shape, window_reach(shape, max_context_len, window, sinks));
    if (route == 0)
        return pa_decode_window_workspace_bytes(shape);
    DeviceInfo* dev;
    return route > 0 && device_info(&dev) == PA_OK
               ? window_split_need(shape, page_size, max_context_len, std::min(window, 1 << 30),
                                   std::min(sinks, 1 << 30), dev)
               : 0;
}

pa_status pa_attention_window(const void* query, const void* key_pages, const void* value_pages,
                              const int32_t* block_table, const int32_t* context_lens,
                              int32_t page_size, float scale, int32_t window, int32_t sinks,
                              void* out, pa_shape shape, int32_t max_context_len, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    if (window <= 0 || sinks < 0 || max_context_len < 0)
        return PA_ERR_INVALID_ARG;
    const int32_t route =
        pa_attention_route(shape, window_reach(shape, max_context_len, window, sinks));
    if (route < 0)
        return PA_ERR_INVALID_ARG;
    if (route == 0)
        return pa_decode_window(query, key_pages, value_pages, block_table, context_lens,
                                page_size, scale, window, sinks, out, shape, max_context_len,
                                workspace, workspace_bytes, stream);
    return run_window_prefill(query, key_pages, value_pages, block_table, context_lens, page_size,
                              scale, window, sinks, out, shape, max_context_len, workspace,
                              workspace_bytes, stream);
}

size_t pa_attention_window_fp8_workspace_bytes(pa_shape shape, int32_t page_size,
                                               int32_t max_context_len, int32_t window,
                                               int32_t sinks)
{
    const int32_t route = route_fp8(shape);
    if (!pow2_in(page_size, 1, 256) || route < 0 || shape.head_dim != 128 || window <= 0 || sinks < 0 || max_context_len < 0)
        return 0;
    if (route == 0)
        return pa_decode_window_workspace_bytes(shape);
    WindowCopyPlan p;
    return plan_window_copy(shape, max_context_len, std::min(window, 1 << 30),
                            std::min(sinks, 1 << 30), &p) == PA_OK
               ? p.total
               : 0;
}

pa_status pa_attention_window_fp8(const void* query, const void* key_pages,
                                  const void* value_pages, const int32_t* block_table,
                                  const int32_t* context_lens, int32_t page_size, float scale,
                                  float k_scale, float v_scale, int32_t window, int32_t sinks,
                                  void* out, pa_shape shape, int32_t max_context_len,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    const int32_t route = route_fp8(shape);
    if (route < 0)
        return PA_ERR_INVALID_ARG;
    if (route == 0)
        return pa_decode_window_fp8(query, key_pages, value_pages, block_table, context_lens,
                                    page_size, scale, k_scale, v_scale, window, sinks, out, shape,
                                    max_context_len, workspace, workspace_bytes, stream);
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    int32_t cut = 0;
    if ((st = check_window(window, sinks, &cut)) != PA_OK)
        return st;
    const int32_t first = std::min(sinks, 1 << 30);
    if (bad_scales(k_scale, v_scale))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    WindowCopyPlan p;
    if ((st = plan_window_copy(shape, max_context_len, cut, first, &p)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < p.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    Fp8PagesArgs c;
    memset(&c, 0, sizeof c);
    c.key_pages = static_cast<const uint8_t*>(key_pages);
    c.value_pages = static_cast<const uint8_t*>(value_pages);
    c.block_table = block_table;
    c.context_lens = context_lens;
    c.key_out = reinterpret_cast<uint16_t*>(w);
    c.value_out = reinterpret_cast<uint16_t*>(w + p.kv_bytes);
    c.table_out = reinterpret_cast<int32_t*>(w + p.table_off);
    c.err = dev->err;
    c.B = shape.batch;
    c.H_kv = shape.num_kv_heads;
    c.ps = page_size;
    c.max_pages = shape.max_pages;
    c.num_pages = shape.num_pages;
    c.P2 = int32_t(p.P2);
    c.P1 = int32_t(p.P1);
    c.window = cut;
    c.sinks = first;
    c.L = shape.q_len;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_fp8_pages_to_bf16(c, s) != cudaSuccess)
        return PA_ERR_CUDA;
    return run_prefill_window(query, c.key_out, c.value_out, c.table_out, context_lens, 128,
                              scale * k_scale, cut, first, v_scale, out, p.copy, max_context_len,
                              w + p.split_off, p.split_bytes, s);
}

size_t pa_decode_weights_workspace_bytes(pa_shape shape, int32_t max_context_len)
{
    WeightPlan p;
    return plan_weights(shape, max_context_len, &p) == PA_OK ? p.total : 0;
}

pa_status pa_decode_weights(const void* query, const void* key_pages, const void* value_pages,
                            float* weight_pages, const int32_t* block_table,
                            const int32_t* context_lens, int32_t page_size, float scale,
                            int causal, float decay, void* out, pa_shape shape,
                            int32_t max_context_len, void* workspace, size_t workspace_bytes,
                            void* stream)
{
    return run_decode_weights(query, key_pages, value_pages, weight_pages, block_table,
                              context_lens, page_size, scale, 0, 1.f, 1.f, causal, decay, out,
                              shape, max_context_len, workspace, workspace_bytes, stream);
}

pa_status pa_decode_weights_fp8(const void* query, const void* key_pages, const void* value_pages,
                                float* weight_pages, const int32_t* block_table,
                                const int32_t* context_lens, int32_t page_size, float scale,
                                float k_scale, float v_scale, int causal, float decay, void* out,
                                pa_shape shape, int32_t max_context_len, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    return run_decode_weights(query, key_pages, value_pages, weight_pages, block_table,
                              context_lens, page_size, scale, 1, k_scale, v_scale, causal, decay,
                              out, shape, max_context_len, workspace, workspace_bytes, stream);
}

pa_status pa_gather_kv(const void* key_pages, const void* value_pages, const int32_t* block_table,
                       const int32_t* context_lens, int32_t page_size, pa_shape shape,
                       int32_t dense_len, void* key_dense, void* value_dense, void* stream)
{
    if (!key_pages || !value_pages || !block_table || !context_lens || !key_dense || !value_dense)
        return PA_ERR_INVALID_ARG;
    if (shape.batch <= 0 || shape.num_kv_heads <= 0 || shape.num_pages <= 0 ||
        shape.max_pages <= 0 || shape.head_dim <= 0 || dense_len <= 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key_pages) || !aligned16(value_pages) || !aligned16(key_dense) ||
        !aligned16(value_dense))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 64 && shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    if (!pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(shape.num_pages) * shape.num_kv_heads * page_size >= (int64_t(1) << 31) ||
        int64_t(shape.max_pages) * page_size >= (int64_t(1) << 30) ||
        2 * int64_t(shape.batch) * shape.num_kv_heads * dense_len * (shape.head_dim / 8) >=
            (int64_t(1) << 40))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    GatherArgs a;
    a.key_pages = static_cast<const uint16_t*>(key_pages);
    a.value_pages = static_cast<const uint16_t*>(value_pages);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.key_dense = static_cast<uint16_t*>(key_dense);
    a.value_dense = static_cast<uint16_t*>(value_dense);
    a.err = dev->err;
    a.B = shape.batch;
    a.H_kv = shape.num_kv_heads;
    a.D = shape.head_dim;
    a.ps = page_size;
    a.num_pages = shape.num_pages;
    a.max_pages = shape.max_pages;
    a.dense_len = dense_len;
    return launch_gather(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                               : PA_ERR_CUDA;
}

namespace {

// Checks of a read-back's sizes.
pa_status check_gather_q4(const pa_shape& s, int32_t page_size)
{
    if (s.batch <= 0 || s.num_kv_heads <= 0 || s.num_pages <= 0 || s.max_pages <= 0 || s.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (s.head_dim != 128 || !pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(s.num_pages) * s.num_kv_heads * page_size >= (int64_t(1) << 31) ||
        int64_t(s.max_pages) * page_size >= (int64_t(1) << 30))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

PageReadArgs page_read_args(const void* key_pages, const void* value_pages, const int32_t* block_table,
                        const int32_t* context_lens, int32_t page_size, const pa_shape& s,
                        const DeviceInfo* dev)
{
    PageReadArgs a;
    memset(&a, 0, sizeof a);
    a.key_pages = static_cast<const uint8_t*>(key_pages);
    a.value_pages = static_cast<const uint8_t*>(value_pages);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_kv = s.num_kv_heads;
    a.ps = page_size;
    a.num_pages = s.num_pages;
    a.max_pages = s.max_pages;
    return a;
}

}  // namespace

pa_status pa_append_kv_q4(const void* key, const void* value, void* key_pages, void* value_pages,
                          const int32_t* slot_mapping, int32_t page_size, pa_shape shape,
                          void* stream)
{
    if (!key || !value || !key_pages || !value_pages || !slot_mapping)
        return PA_ERR_INVALID_ARG;
    if (shape.batch <= 0 || shape.num_kv_heads <= 0 || shape.q_len < 0 || shape.num_pages <= 0 ||
        shape.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_pages) || !aligned16(value_pages))
        return PA_ERR_INVALID_ARG;
    if (shape.head_dim != 128 || !pow2_in(page_size, 1, 256))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(shape.num_pages) * shape.num_kv_heads * page_size >= (int64_t(1) << 31) ||
        int64_t(shape.batch) * shape.q_len * shape.num_kv_heads >= (int64_t(1) << 31) - 65536 * 16)
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (shape.q_len == 0)
        return PA_OK;
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.key = static_cast<const uint16_t*>(key);
    a.value = static_cast<const uint16_t*>(value);
    a.key_pages = static_cast<uint16_t*>(key_pages);     // byte pages; the kernel casts back
    a.value_pages = static_cast<uint16_t*>(value_pages);
    a.slot_mapping = slot_mapping;
    a.err = dev->err;
    a.B = shape.batch;
    a.L_new = shape.q_len;
    a.H_kv = shape.num_kv_heads;
    a.D = 128;
    a.ps = page_size;
    a.num_pages = shape.num_pages;
    return launch_append_q4(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                  : PA_ERR_CUDA;
}

pa_status pa_gather_kv_q4(const void* key_pages, const void* value_pages,
                          const int32_t* block_table, const int32_t* context_lens,
                          int32_t page_size, pa_shape shape, int32_t dense_len, void* key_dense,
                          void* value_dense, void* stream)
{
    if (!key_pages || !value_pages || !block_table || !context_lens || !key_dense || !value_dense ||
        dense_len <= 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key_pages) || !aligned16(value_pages) || !aligned16(key_dense) ||
        !aligned16(value_dense))
        return PA_ERR_INVALID_ARG;
    pa_status st = check_gather_q4(shape, page_size);
    if (st != PA_OK)
        return st;
    if (int64_t(shape.batch) * shape.num_kv_heads * ((int64_t(dense_len) + 127) / 128) >=
        (int64_t(1) << 31))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    PageReadArgs a = page_read_args(key_pages, value_pages, block_table, context_lens, page_size, shape, dev);
    a.key_out = static_cast<uint16_t*>(key_dense);
    a.value_out = static_cast<uint16_t*>(value_dense);
    a.head_stride = int64_t(dense_len) * 128;
    a.batch_stride = a.head_stride * shape.num_kv_heads;
    a.block_stride = int64_t(kCopyPageRows) * 128;
    a.max_len = dense_len;
    return launch_read_pages(a, kQ4Pool, 128, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

namespace {

// bf16 copies, in pages of 128 tokens, of what `s.batch` tables lead to: K and V (kv_bytes
// each; V of 4-bit pools in f16), then the copies' table (P2 entries each) table_off bytes
// into w.
pa_status copy_pages(const void* key_pages, const void* value_pages, const int32_t* block_table,
                     const int32_t* context_lens, int32_t page_size, const pa_shape& s, int kind,
                     int64_t P2, size_t kv_bytes, size_t table_off, const DeviceInfo* dev, uint8_t* w,
                     cudaStream_t stream)
{
    PageReadArgs a = page_read_args(key_pages, value_pages, block_table, context_lens, page_size, s, dev);
    a.key_out = reinterpret_cast<uint16_t*>(w);
    a.value_out = reinterpret_cast<uint16_t*>(w + kv_bytes);
    a.table_out = reinterpret_cast<int32_t*>(w + table_off);
    a.head_stride = int64_t(kCopyPageRows) * s.head_dim;
    a.block_stride = a.head_stride * s.num_kv_heads;
    a.batch_stride = a.block_stride * P2;
    a.max_len = int32_t(P2 * kCopyPageRows);
    a.copy_pages = int32_t(P2);
    a.f16_values = kind == kQ4Pool;
    return launch_read_pages(a, kind, s.head_dim, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// What the few-row kernel takes of a call (no tensor maps, no outputs of its modes).
DecodeArgs rows_args(const void* query, const int32_t* block_table, const int32_t* context_lens,
                     int32_t page_size, float scale, int causal, void* out, const pa_shape& s, int kind,
                     DecodeMode mode, const DeviceInfo* dev)
{
    DecodeArgs a;
    memset(&a, 0, sizeof a);
    a.q = static_cast<const uint16_t*>(query);
    a.out = static_cast<uint16_t*>(out);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.err = dev->err;
    a.B = s.batch;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.L = s.q_len;
    a.D = s.head_dim;
    a.ps = page_size;
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.G = s.num_q_heads / s.num_kv_heads;
    a.R = a.G * s.q_len;
    a.box_rows = decode_rows_box(s, kind, page_size);
    a.swz = a.box_rows >= 8 ? 7 : 0;
    while ((1 << a.ps_shift) < page_size)
        ++a.ps_shift;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = causal ? 1 : 0;
    a.fp8 = kind == kE4m3Pool ? 1 : 0;
    a.v_scale = 1.f;
    a.mode = mode;
    return a;
}

// Tiles of keys by four, at most, of all segments of the few-row kernel.
int64_t rows_granules(const pa_shape& s, int kind, int64_t keys)
{
    const int64_t MS = (int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len + kSegmentRows - 1) / kSegmentRows;
    const int64_t tile = 4 * decode_rows_tile(s, kind);
    return int64_t(s.batch) * s.num_kv_heads * MS * std::max<int64_t>(1, (keys + tile - 1) / tile);
}

// Whether there are at most kMaxSegments segments, and the granules of the longest contexts
// that the tables have room for can be counted in 32 bits, as the few-row kernel does.
bool rows_count_ok(const pa_shape& s, int kind, int32_t page_size)
{
    const int64_t bh = int64_t(s.batch) * s.num_kv_heads;
    const int64_t MS = (int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len + kSegmentRows - 1) / kSegmentRows;
    return bh <= kMaxSegments && bh * MS <= kMaxSegments &&
           rows_granules(s, kind, int64_t(s.max_pages) * page_size) < (int64_t(1) << 31);
}

bool rows_shape_ok(const pa_shape& s)
{
    return s.batch > 0 && s.num_q_heads > 0 && s.num_kv_heads > 0 && s.q_len > 0 &&
           s.num_q_heads % s.num_kv_heads == 0 &&
           int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len < (int64_t(1) << 30);
}

}  // namespace

size_t pa_decode_q4_workspace_bytes(pa_shape shape)
{
    DeviceInfo* dev;
    if (!rows_shape_ok(shape) || shape.head_dim != 128 || device_info(&dev) != PA_OK ||
        !decode_rows_fits(shape, kQ4Pool, kFull, dev->max_smem_optin))
        return 0;
    return decode_rows_workspace_bytes(shape, kQ4Pool, kFull, dev->sm_count);
}

pa_status pa_decode_q4(const void* query, const void* key_pages, const void* value_pages,
                       const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                       float scale, int causal, void* out, pa_shape shape, int32_t max_context_len,
                       void* workspace, size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (shape.head_dim != 128 || !rows_shape_ok(shape) || !rows_count_ok(shape, kQ4Pool, page_size))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    if (!decode_rows_fits(shape, kQ4Pool, kFull, dev->max_smem_optin))
        return PA_ERR_UNSUPPORTED;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
        workspace_bytes < decode_rows_workspace_bytes(shape, kQ4Pool, kFull, dev->sm_count))
        return PA_ERR_WORKSPACE;
    DecodeArgs a = rows_args(query, block_table, context_lens, page_size, scale, causal, out, shape, kQ4Pool,
                             kFull, dev);
    a.key_rows = static_cast<const uint8_t*>(key_pages);
    a.value_rows = static_cast<const uint8_t*>(value_pages);
    const int grid = decode_rows_launch_grid(
        shape, kQ4Pool, kFull, max_context_len > 0 ? rows_granules(shape, kQ4Pool, max_context_len) : 0, dev->sm_count);
    const CUtensorMap none = {};
    return launch_decode_rows(none, none, a, shape, kQ4Pool, grid, workspace, dev->id,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t pa_prefill_q4_workspace_bytes(pa_shape shape, int32_t max_context_len)
{
    return pa_prefill_fp8_workspace_bytes(shape, max_context_len);
}

pa_status pa_prefill_q4(const void* query, const void* key_pages, const void* value_pages,
                        const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                        float scale, int causal, void* out, pa_shape shape,
                        int32_t max_context_len, void* workspace, size_t workspace_bytes,
                        void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (shape.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    Fp8PrefillPlan p;
    if ((st = plan_prefill_fp8(shape, max_context_len, dev, &p)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < p.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = copy_pages(key_pages, value_pages, block_table, context_lens, page_size, shape, kQ4Pool, p.P2,
                         p.kv_bytes, p.table_off, dev, w, s)) != PA_OK)
        return st;
    return run_prefill_tc(query, w, w + p.kv_bytes, reinterpret_cast<int32_t*>(w + p.table_off),
                          context_lens, 128, scale, causal, out, p.copy, s,
                          p.split_bytes ? w + p.split_off : nullptr, p.split_bytes, 1.f,
                          p.piece_bytes ? w + p.split_off : nullptr, p.piece_bytes, true);
}

namespace {

// Route of pa_attention_q4: the few-row kernel reads K and V once per 16 rows of a
// (request, KV head), the prefill copies them first. With 1, 4, 7 and 8 query heads a KV
// head, us: 16 requests of 1000-4000 keys, L = 8: few rows 21, 45, 44, 80, prefill 75, 96,
// 82, 147; 4 of 8000-16000: 25, 52, 51, 90 and 190, 137, 117, 204. (At L = 9 to 16 few rows
// are still ahead, or level: 28, 80, 71, 148 at 16. The limit is pa_attention_fp8's, so that a
// chunk goes the same way over either pool.)
int32_t route_q4(const pa_shape& shape) { return shape.q_len <= 0 ? -1 : shape.q_len <= 8 ? 0 : 1; }

}  // namespace

size_t pa_attention_q4_workspace_bytes(pa_shape shape, int32_t max_context_len)
{
    const int32_t route = route_q4(shape);
    if (route < 0)
        return 0;
    return route == 0 ? pa_decode_q4_workspace_bytes(shape)
                      : pa_prefill_q4_workspace_bytes(shape, max_context_len);
}

pa_status pa_attention_q4(const void* query, const void* key_pages, const void* value_pages,
                          const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                          float scale, int causal, void* out, pa_shape shape,
                          int32_t max_context_len, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    const int32_t route = route_q4(shape);
    if (route < 0)
        return PA_ERR_INVALID_ARG;
    return (route == 0 ? pa_decode_q4 : pa_prefill_q4)(
        query, key_pages, value_pages, block_table, context_lens, page_size, scale, causal, out, shape,
        max_context_len, workspace, workspace_bytes, stream);
}

namespace {

// A decode behind shared prefixes: whether the prefixes are attended to on copies (bf16
// pages too small for the prefix kernel's TMA boxes), and the workspace: copies with their
// table, the prefixes' states, the notes for the merge, the few-row kernel's states.
struct PrefixPlan {
    bool copies = false;
    int64_t P2 = 0;
    int prefix_grid = 0;
    int32_t items = 0;
    size_t kv_bytes = 0, table_off = 0, state_off = 0, ml_off = 0, pieces_off = 0, note_off = 0, rows_off = 0,
           total = 0;
};

pa_status plan_prefix(const pa_shape& s, int32_t page_size, int kind, int32_t count, int32_t max_prefix_len,
                      const DeviceInfo* dev, PrefixPlan* p)
{
    if (s.batch <= 0 || s.num_q_heads <= 0 || s.num_kv_heads <= 0 || s.q_len <= 0 || s.head_dim <= 0 ||
        count <= 0 || max_prefix_len <= 0)
        return PA_ERR_INVALID_ARG;
    if ((s.head_dim != 128 && (kind != kBf16Pool || s.head_dim != 64)) || !pow2_in(page_size, 1, 256) ||
        !rows_shape_ok(s) || !rows_count_ok(s, kind, page_size) || count > kMaxPrefixes ||
        max_prefix_len >= (1 << 30))
        return PA_ERR_UNSUPPORTED;
    const int64_t R = int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len;
    if (!decode_rows_fits(s, kind, kSuffix, dev->max_smem_optin) || s.batch * R >= (int64_t(1) << 30) ||
        s.batch * R * s.num_kv_heads >= (int64_t(1) << 31) ||
        prefix_smem_bytes(s.head_dim, kind, count) > size_t(dev->max_smem_optin))
        return PA_ERR_UNSUPPORTED;
    p->copies = kind == kBf16Pool && page_size < 8;
    p->P2 = (int64_t(max_prefix_len) + kCopyPageRows - 1) / kCopyPageRows;
    if (p->copies) {
        const int64_t pages = count * p->P2;
        if (pages * s.num_kv_heads * kCopyPageRows >= (int64_t(1) << 31))
            return PA_ERR_UNSUPPORTED;
        p->kv_bytes = size_t(pages) * s.num_kv_heads * kCopyPageRows * s.head_dim * 2;
        p->table_off = 2 * p->kv_bytes;
        p->state_off = (p->table_off + size_t(pages) * 4 + 255) & ~size_t(255);
    }
    // at most a block an SM and a block a tile (Ranges leaves some without work where items
    // are few and short)
    const int64_t items = s.num_kv_heads * (s.batch * R / 256 + count);
    p->prefix_grid = int(std::min<int64_t>(dev->sm_count, items * p->P2));
    if (items * prefix_item_units(p->P2) >= (int64_t(1) << 31))   // units are 32-bit numbers
        return PA_ERR_UNSUPPORTED;
    p->items = int32_t(items);
    size_t ml = 0, pieces = 0;
    const size_t states = prefix_state_bytes(s, items, p->prefix_grid, &ml, &pieces);
    p->ml_off = p->state_off + ml;
    p->pieces_off = p->state_off + pieces;
    // notes for the merge: an int4 a row, an int2 a segment
    const int64_t segments = int64_t(s.batch) * s.num_kv_heads * ((R + kSegmentRows - 1) / kSegmentRows);
    p->note_off = (p->state_off + states + 255) & ~size_t(255);
    p->rows_off = (p->note_off + size_t(s.batch * R) * s.num_kv_heads * 16 + size_t(segments) * 8 + 255) & ~size_t(255);
    p->total = p->rows_off + decode_rows_workspace_bytes(s, kind, kSuffix, dev->sm_count);
    return PA_OK;
}

size_t prefix_workspace(const pa_shape& s, int32_t page_size, int kind, int32_t count, int32_t max_prefix_len)
{
    DeviceInfo* dev;
    PrefixPlan p;
    if (device_info(&dev) != PA_OK || plan_prefix(s, page_size, kind, count, max_prefix_len, dev, &p) != PA_OK)
        return 0;
    return p.total;
}

pa_status run_decode_prefix(const void* query, const void* key_pages, const void* value_pages,
                            const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                            float scale, int kind, float k_scale, float v_scale, const int32_t* prefix_table,
                            const int32_t* prefix_lens, const int32_t* prefix_starts, int32_t num_prefixes,
                            int32_t prefix_pages, int32_t max_prefix_len, void* out, const pa_shape& shape,
                            int32_t max_context_len, void* workspace, size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                                   out, shape);
    if (st != PA_OK)
        return st;
    if (!prefix_table || !prefix_lens || !prefix_starts || prefix_pages <= 0 ||
        (kind == kE4m3Pool && bad_scales(k_scale, v_scale)))
        return PA_ERR_INVALID_ARG;
    if (int64_t(prefix_pages) * page_size >= (int64_t(1) << 30) || !rows_shape_ok(shape) ||
        !rows_count_ok(shape, kind, page_size))
        return PA_ERR_UNSUPPORTED;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    PrefixPlan p;
    if ((st = plan_prefix(shape, page_size, kind, num_prefixes, max_prefix_len, dev, &p)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < p.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int D = shape.head_dim;

    PrefixKernelArgs a;
    memset(&a, 0, sizeof a);
    a.q = static_cast<const uint16_t*>(query);
    a.context_lens = context_lens;
    a.state = reinterpret_cast<float*>(w + p.state_off);
    a.state_ml = reinterpret_cast<float2*>(w + p.ml_off);
    a.more_pieces = w + p.pieces_off;
    a.most_items = p.items;
    a.note_row = reinterpret_cast<int4*>(w + p.note_off);
    a.err = dev->err;
    a.prefix.table = prefix_table;
    a.prefix.lens = prefix_lens;
    a.prefix.starts = prefix_starts;
    a.prefix.count = num_prefixes;
    a.prefix.pages = prefix_pages;
    a.prefix.cap = int32_t(std::min<int64_t>(int64_t(prefix_pages) * page_size, max_prefix_len));
    a.B = shape.batch;
    a.H_q = shape.num_q_heads;
    a.H_kv = shape.num_kv_heads;
    a.L = shape.q_len;
    a.G = shape.num_q_heads / shape.num_kv_heads;
    a.R = a.G * shape.q_len;
    a.ps = page_size;
    a.num_pages = shape.num_pages;
    a.block_ps = page_size;
    a.max_pages = shape.max_pages;
    a.scale_log2 = scale * 1.4426950408889634f * k_scale;
    const PrefixArgs own_table = a.prefix;
    const void *kp = key_pages, *vp = value_pages;
    pa_shape pool = shape;
    if (p.copies) {
        kp = w;
        vp = w + p.kv_bytes;
        a.prefix.table = reinterpret_cast<const int32_t*>(w + p.table_off);
        a.prefix.pages = int32_t(p.P2);
        a.ps = kCopyPageRows;
        a.num_pages = pool.num_pages = int32_t(num_prefixes * p.P2);
    }
    a.box_rows = std::min(a.ps, 128);
    const uint64_t pool_rows = uint64_t(pool.num_pages) * shape.num_kv_heads * a.ps;
    CUtensorMap kmap = {}, vmap = {};
    if (kind == kBf16Pool &&
        ((st = encode_rows_map(&kmap, kp, pool_rows, uint32_t(a.box_rows), uint32_t(D))) != PA_OK ||
         (st = encode_rows_map(&vmap, vp, pool_rows, uint32_t(a.box_rows), uint32_t(D))) != PA_OK))
        return st;
    a.key_rows = static_cast<const uint8_t*>(key_pages);
    a.value_rows = static_cast<const uint8_t*>(value_pages);
    while ((1 << a.ps_shift) < a.ps)
        ++a.ps_shift;
    a.by_R.set(a.R);
    a.by_L.set(a.L);
    a.by_H.set(a.H_kv);

    DecodeArgs d = rows_args(query, block_table, context_lens, page_size, scale * k_scale, 1, out, shape, kind,
                             kSuffix, dev);
    d.key_rows = static_cast<const uint8_t*>(key_pages);
    d.value_rows = static_cast<const uint8_t*>(value_pages);
    d.prefix = own_table;
    d.note_segment = reinterpret_cast<int2*>(a.note_row + int64_t(a.B) * a.H_kv * a.R);
    CUtensorMap skmap = {}, svmap = {};
    if (kind != kQ4Pool &&
        ((st = encode_pool_map(&skmap, key_pages, shape, page_size, kind == kE4m3Pool, d.box_rows)) != PA_OK ||
         (st = encode_pool_map(&svmap, value_pages, shape, page_size, kind == kE4m3Pool, d.box_rows)) != PA_OK))
        return st;
    // From here on only a launch can fail.
    const cudaError_t e = prepare_prefix(D, kind, dev->id);
    if (e != cudaSuccess)
        return e == cudaErrorNotSupported ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
    if (p.copies) {
        pa_shape tables = shape;
        tables.batch = num_prefixes;
        tables.max_pages = prefix_pages;
        if ((st = copy_pages(key_pages, value_pages, prefix_table, prefix_lens, page_size, tables, kind, p.P2,
                             p.kv_bytes, p.table_off, dev, w, s)) != PA_OK)
            return st;
    }
    if (launch_prefix(kmap, vmap, a, D, kind, p.prefix_grid, s) != cudaSuccess)
        return PA_ERR_CUDA;
    const int grid = decode_rows_launch_grid(
        shape, kind, kSuffix, max_context_len > 0 ? rows_granules(shape, kind, max_context_len) : 0, dev->sm_count);
    if (launch_decode_rows(skmap, svmap, d, shape, kind, grid, w + p.rows_off, dev->id, s) != cudaSuccess)
        return PA_ERR_CUDA;

    PrefixMergeArgs m;
    memset(&m, 0, sizeof m);
    m.prefix_args = a;
    m.suffix_state = reinterpret_cast<const float*>(w + p.rows_off);
    m.out = static_cast<uint16_t*>(out);
    m.out_scale = v_scale;
    m.note_segment = d.note_segment;
    m.MS = (a.R + kSegmentRows - 1) / kSegmentRows;
    m.row_tiles = decode_rows_row_tiles(shape);
    return launch_prefix_merge(m, D, dev->sm_count, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

size_t pa_decode_prefix_workspace_bytes(pa_shape shape, int32_t page_size, int32_t num_prefixes,
                                        int32_t max_prefix_len)
{
    return prefix_workspace(shape, page_size, kBf16Pool, num_prefixes, max_prefix_len);
}

size_t pa_decode_prefix_fp8_workspace_bytes(pa_shape shape, int32_t page_size, int32_t num_prefixes,
                                            int32_t max_prefix_len)
{
    return prefix_workspace(shape, page_size, kE4m3Pool, num_prefixes, max_prefix_len);
}

size_t pa_decode_prefix_q4_workspace_bytes(pa_shape shape, int32_t page_size, int32_t num_prefixes,
                                           int32_t max_prefix_len)
{
    return prefix_workspace(shape, page_size, kQ4Pool, num_prefixes, max_prefix_len);
}

pa_status pa_decode_prefix(const void* query, const void* key_pages, const void* value_pages,
                           const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                           float scale, const int32_t* prefix_table, const int32_t* prefix_lens,
                           const int32_t* prefix_starts, int32_t num_prefixes, int32_t prefix_pages,
                           int32_t max_prefix_len, void* out, pa_shape shape, int32_t max_context_len,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    return run_decode_prefix(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                             kBf16Pool, 1.f, 1.f, prefix_table, prefix_lens, prefix_starts, num_prefixes,
                             prefix_pages, max_prefix_len, out, shape, max_context_len, workspace,
                             workspace_bytes, stream);
}

pa_status pa_decode_prefix_fp8(const void* query, const void* key_pages, const void* value_pages,
                               const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                               float scale, float k_scale, float v_scale, const int32_t* prefix_table,
                               const int32_t* prefix_lens, const int32_t* prefix_starts,
                               int32_t num_prefixes, int32_t prefix_pages, int32_t max_prefix_len, void* out,
                               pa_shape shape, int32_t max_context_len, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    return run_decode_prefix(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                             kE4m3Pool, k_scale, v_scale, prefix_table, prefix_lens, prefix_starts,
                             num_prefixes, prefix_pages, max_prefix_len, out, shape, max_context_len, workspace,
                             workspace_bytes, stream);
}

pa_status pa_decode_prefix_q4(const void* query, const void* key_pages, const void* value_pages,
                              const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                              float scale, const int32_t* prefix_table, const int32_t* prefix_lens,
                              const int32_t* prefix_starts, int32_t num_prefixes, int32_t prefix_pages,
                              int32_t max_prefix_len, void* out, pa_shape shape, int32_t max_context_len,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    return run_decode_prefix(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                             kQ4Pool, 1.f, 1.f, prefix_table, prefix_lens, prefix_starts, num_prefixes,
                             prefix_pages, max_prefix_len, out, shape, max_context_len, workspace,
                             workspace_bytes, stream);
}

pa_status pa_decode_dense(const void* query, const void* key_dense, const void* value_dense,
                          const int32_t* context_lens, int32_t dense_len, float scale, int causal,
                          void* out, pa_shape shape, int32_t max_context_len, void* workspace,
                          size_t workspace_bytes, void* stream)
{
    if (dense_len < 64 || dense_len % 64 != 0)
        return PA_ERR_UNSUPPORTED;
    // The dense buffers are a pool of B pages of dense_len tokens, request b
    // in page b (the kernel does not read a block table for them).
    pa_shape s = shape;
    s.num_pages = shape.batch;
    s.max_pages = 1;
    if (!query || !key_dense || !value_dense || !context_lens || !out)
        return PA_ERR_INVALID_ARG;
    if (s.batch <= 0 || s.num_q_heads <= 0 || s.num_kv_heads <= 0 || s.q_len <= 0 ||
        s.head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query) || !aligned16(key_dense) || !aligned16(value_dense) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    if (s.head_dim != 64 && s.head_dim != 128)
        return PA_ERR_UNSUPPORTED;
    if (s.num_q_heads % s.num_kv_heads != 0)
        return PA_ERR_UNSUPPORTED;
    if (int64_t(s.batch) * s.num_kv_heads * dense_len >= (int64_t(1) << 31) ||
        int64_t(dense_len) >= (int64_t(1) << 30))
        return PA_ERR_UNSUPPORTED;
    return run_split_kv(query, key_dense, value_dense, nullptr, context_lens, dense_len, scale,
                        causal, out, s, max_context_len, workspace, workspace_bytes, 0,
                        static_cast<cudaStream_t>(stream), 1);
}

namespace {

// pa_prefill; piece_ws: room for the pairs kernel's tail pieces (pa_attention's
// workspace), or null.
pa_status prefill_route(const void* query, const void* key_pages, const void* value_pages,
                        const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                        float scale, int causal, void* out, pa_shape shape, void* stream,
                        void* piece_ws, size_t piece_ws_bytes)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    if (shape.head_dim == 128 || shape.head_dim == 64) {
        st = run_prefill_tc(query, key_pages, value_pages, block_table, context_lens, page_size,
                            scale, causal, out, shape, static_cast<cudaStream_t>(stream), nullptr, 0,
                            1.f, piece_ws, piece_ws_bytes);
        if (st != PA_ERR_UNSUPPORTED || shape.head_dim == 128)
            return st;
    }
    // Without the pairs kernel's register split (head_dim 64, or pages of
    // fewer than 8 tokens): the split-KV kernel with whole segments per block.
    return run_split_kv(query, key_pages, value_pages, block_table, context_lens, page_size,
                        scale, causal, out, shape, 0, nullptr, 0, 1,
                        static_cast<cudaStream_t>(stream));
}

}  // namespace

pa_status pa_prefill(const void* query, const void* key_pages, const void* value_pages,
                     const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                     float scale, int causal, void* out, pa_shape shape, void* stream)
{
    return prefill_route(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                         causal, out, shape, stream, nullptr, 0);
}

size_t pa_prefill_workspace_bytes(pa_shape shape, int32_t page_size)
{
    DeviceInfo* dev;
    if (device_info(&dev) != PA_OK)
        return 0;
    return split_prefill_need(shape, page_size, dev);
}

pa_status pa_prefill_split(const void* query, const void* key_pages, const void* value_pages,
                           const int32_t* block_table, const int32_t* context_lens,
                           int32_t page_size, float scale, int causal, void* out, pa_shape shape,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    pa_status st = check_attention(query, key_pages, value_pages, block_table, context_lens,
                                   page_size, scale, out, shape);
    if (st != PA_OK)
        return st;
    DeviceInfo* dev;
    if ((st = device_info(&dev)) != PA_OK)
        return st;
    const size_t need = split_prefill_need(shape, page_size, dev);
    if (need == 0)   // another prefill kernel serves this shape; no workspace used
        return pa_prefill(query, key_pages, value_pages, block_table, context_lens, page_size,
                          scale, causal, out, shape, stream);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_WORKSPACE;
    return run_prefill_tc(query, key_pages, value_pages, block_table, context_lens, page_size,
                          scale, causal, out, shape, static_cast<cudaStream_t>(stream), workspace,
                          workspace_bytes);
}

int32_t pa_attention_route(pa_shape shape, int32_t max_context_len)
{
    if (shape.q_len <= 0 || shape.num_q_heads <= 0 || shape.num_kv_heads <= 0)
        return -1;
    // The split-KV decode reads a KV group's K/V once per 64 of its query
    // rows (four 16-row tiles per segment) and its cost grows with the rows;
    // the persistent tile prefill pays a fixed cost per 128-row tile.
    // Measured crossover on GB300 (32 requests, contexts of 1k to 4k tokens,
    // page size 16, 1, 4 and 7 query heads per KV group): decode is faster up
    // to 24 rows per request (within 3 % at 1k contexts), the two tie at 32
    // rows from about 3k-token contexts on, and prefill is faster beyond.
    return shape.q_len <= 24 || (shape.q_len <= 32 && max_context_len >= 3072) ? 0 : 1;
}

pa_status pa_attention(const void* query, const void* key_pages, const void* value_pages,
                       const int32_t* block_table, const int32_t* context_lens, int32_t page_size,
                       float scale, int causal, void* out, pa_shape shape,
                       int32_t max_context_len, void* workspace, size_t workspace_bytes,
                       void* stream)
{
    const int32_t route = pa_attention_route(shape, max_context_len);
    if (route < 0)
        return PA_ERR_INVALID_ARG;
    if (route == 0)
        return pa_decode(query, key_pages, value_pages, block_table, context_lens, page_size,
                         scale, causal, out, shape, max_context_len, workspace, workspace_bytes,
                         stream);
    if (workspace && t_prefill_variant != 4 && t_prefill_variant != 5) {
        // The split kernel pays for its balance at every piece boundary; it
        // is the faster one when the (request, head pair, query tile) items
        // are too few to fill the SMs in whole waves (measured: 1.75x on one
        // 512-row chunk after a 16k prefix, 64 items; equal at 1.7 items per
        // SM; slower beyond).
        DeviceInfo* dev;
        pa_status st = device_info(&dev);
        if (st != PA_OK)
            return st;
        const size_t need = split_prefill_need(shape, page_size, dev);
        const int64_t items = prefill_pair_items(shape);
        if (need > 0 && workspace_bytes >= need && 2 * items < 3 * int64_t(dev->sm_count) &&
            (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0)
            return pa_prefill_split(query, key_pages, value_pages, block_table, context_lens,
                                    page_size, scale, causal, out, shape, workspace,
                                    workspace_bytes, stream);
    }
    // the pairs kernel, which balances one to two items per block with tail
    // pieces in the workspace
    return prefill_route(query, key_pages, value_pages, block_table, context_lens, page_size, scale,
                         causal, out, shape, stream, workspace, workspace_bytes);
}

pa_status pa_get_device_error(void* stream, uint32_t* flags)
{
    DeviceInfo* dev;
    pa_status st = device_info(&dev);
    if (st != PA_OK)
        return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return PA_ERR_CUDA;
    unsigned v = 0;
    const unsigned zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess)
        return PA_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero) != cudaSuccess)
        return PA_ERR_CUDA;
    if (flags)
        *flags = v;
    if (v & PA_DEVERR_TIMEOUT)
        return PA_ERR_DEVICE_TIMEOUT;
    return v ? PA_ERR_DEVICE_BOUNDS : PA_OK;
}

const char* pa_status_string(pa_status status)
{
    switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG: invalid argument";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: unsupported shape or page size";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: workspace missing, too small or misaligned";
    case PA_ERR_NO_PAGES: return "PA_ERR_NO_PAGES: page pool or block-table row full (nothing changed)";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: CUDA call or launch failed";
    case PA_ERR_DEVICE_BOUNDS: return "PA_ERR_DEVICE_BOUNDS: kernel met an out-of-range index";
    case PA_ERR_DEVICE_TIMEOUT: return "PA_ERR_DEVICE_TIMEOUT: kernel wait gave up";
    }
    return "unknown pa_status";
}

const char* pa_version(void) { return "0.1.0"; }

void pa_debug_arm_wait_timeout(void) { t_arm_unset_wait = true; }

int pa_debug_prefill_variant(int variant)
{
    const int prev = t_prefill_variant;
    t_prefill_variant = (variant == 1 || variant == 2 || variant == 4 || variant == 5 ||
                         variant == 6 || variant == 7)
                            ? variant
                            : 0;
    return prev;
}

}  // extern "C"
