// The few-row kernel (pa_decode_rows.cuh): its instances with a sliding window and with
// the scores kept, and the launch of all of them.
#include "pa_decode_rows.cuh"

#include <atomic>

namespace pa {
namespace rows {
namespace {

template <int D, int KIND, int NT>
Kernels of_mode(int mode)
{
    return mode == kWindow ? kernels_of<D, KIND, NT, kWindow>() : kernels_of<D, KIND, NT, kScores>();
}

Kernels kernels_for(int D, int kind, int NT, int mode)
{
    if (mode == kSuffix)
        return suffix_kernels(D, kind, NT);
    if (kind == kQ4Pool)
        return q4_kernels(NT);
    if (kind == kE4m3Pool)
        return NT == 1 ? of_mode<128, kE4m3Pool, 1>(mode) : of_mode<128, kE4m3Pool, 2>(mode);
    if (D == 64)
        return NT == 1 ? of_mode<64, kBf16Pool, 1>(mode) : of_mode<64, kBf16Pool, 2>(mode);
    return NT == 1 ? of_mode<128, kBf16Pool, 1>(mode) : of_mode<128, kBf16Pool, 2>(mode);
}

// What the launch needs of an instance.
struct Facts {
    size_t slab;                  // bytes of a state
    size_t smem;
    int blocks_per_sm;
};
template <int D, int KIND, int NT>
Facts facts_of(int B, int mode)
{
    using Suffix = Smem<D, KIND, NT, kSuffix>;
    using Other = Smem<D, KIND, NT, kFull>;
    if (mode == kSuffix)
        return {size_t(suffix_slot_floats(D, NT)) * 4, Suffix::bytes(B), Suffix::kBlocksPerSM};
    return {size_t(Other::kSlab), Other::bytes(B), Other::kBlocksPerSM};
}
Facts facts(int D, int kind, int NT, int B, int mode)
{
    if (kind == kQ4Pool)
        return NT == 1 ? facts_of<128, kQ4Pool, 1>(B, mode) : facts_of<128, kQ4Pool, 2>(B, mode);
    if (kind == kE4m3Pool)
        return NT == 1 ? facts_of<128, kE4m3Pool, 1>(B, mode) : facts_of<128, kE4m3Pool, 2>(B, mode);
    if (D == 64)
        return NT == 1 ? facts_of<64, kBf16Pool, 1>(B, mode) : facts_of<64, kBf16Pool, 2>(B, mode);
    return NT == 1 ? facts_of<128, kBf16Pool, 1>(B, mode) : facts_of<128, kBf16Pool, 2>(B, mode);
}

int64_t rows_of(const pa_shape& s) { return int64_t(s.num_q_heads / s.num_kv_heads) * s.q_len; }
int row_tiles(const pa_shape& s) { return rows_of(s) <= 8 ? 1 : 2; }

}  // namespace
}  // namespace rows

bool decode_rows_takes(const pa_shape& s, int max_smem)
{
    // e4m3 and bf16 rings have one size
    return rows::rows_of(s) <= 16 &&
           rows::facts(s.head_dim, kBf16Pool, rows::row_tiles(s), s.batch, kWindow).smem <= size_t(max_smem);
}

bool decode_rows_fits(const pa_shape& s, int kind, int mode, int max_smem)
{
    const int64_t MS = (rows::rows_of(s) + kSegmentRows - 1) / kSegmentRows;
    return int64_t(s.batch) * s.num_kv_heads * MS <= kMaxSegments &&
           rows::facts(s.head_dim, kind, rows::row_tiles(s), s.batch, mode).smem <= size_t(max_smem);
}

int decode_rows_grid(const pa_shape& s, int kind, int mode, int sm_count)
{
    return sm_count * rows::facts(s.head_dim, kind, rows::row_tiles(s), 1, mode).blocks_per_sm;
}

int decode_rows_box(const pa_shape& s, int kind, int page_size)
{
    const int tok = decode_rows_tile(s, kind);
    return page_size < tok ? page_size : tok;
}

size_t decode_rows_workspace_bytes(const pa_shape& s, int kind, int mode, int sm_count)
{
    const int64_t MS = (rows::rows_of(s) + kSegmentRows - 1) / kSegmentRows;
    return (size_t(s.batch) * s.num_kv_heads * size_t(MS) + size_t(decode_rows_grid(s, kind, mode, sm_count))) *
           rows::facts(s.head_dim, kind, rows::row_tiles(s), 1, mode).slab;
}

int decode_rows_tile(const pa_shape& s, int kind) { return kind == kBf16Pool && s.head_dim == 128 ? 16 : 32; }

int decode_rows_row_tiles(const pa_shape& s) { return rows::row_tiles(s); }

int decode_rows_launch_grid(const pa_shape& s, int kind, int mode, int64_t granule_bound, int sm_count)
{
    int64_t grid = decode_rows_grid(s, kind, mode, sm_count);
    // Few granules: two of them a block at least, so that a segment's pieces stay
    // few (one request, window 4096: 11.3 us, 14.0 with one; window 512: 8.4 and 8.2).
    if (granule_bound > 0 && granule_bound < 2 * grid)
        grid = (granule_bound + 2 - 1) / 2;
    return int(grid);
}

cudaError_t launch_decode_rows(const CUtensorMap& key_map, const CUtensorMap& value_map, DecodeArgs a,
                               const pa_shape& s, int kind, int grid, void* workspace, int device,
                               cudaStream_t stream)
{
    const int NT = rows::row_tiles(s);
    a.partials = static_cast<float*>(workspace);
    a.MS = int32_t((a.R + kSegmentRows - 1) / kSegmentRows);
    const rows::Kernels kern = rows::kernels_for(a.D, kind, NT, a.mode);
    constexpr int kMaxDev = 64;
    static std::atomic<bool> raised[kMaxDev][4][2][4];     // pool and head_dim, row tiles, mode
    if (device < 0 || device >= kMaxDev)
        return cudaErrorInvalidDevice;
    const int which = kind == kBf16Pool ? (a.D == 64 ? 0 : 1) : kind == kE4m3Pool ? 2 : 3;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern.main), &raised[device][which][NT - 1][a.mode]);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(rows::kThreads);
    cfg.dynamicSmemBytes = rows::facts(a.D, kind, NT, a.B, a.mode).smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern.main, key_map, value_map, a);
    if (e != cudaSuccess || !kern.merge)
        return e;
    cfg.gridDim = dim3(unsigned(int64_t(a.B) * a.H_kv * (a.mode == kFull ? a.MS : 1)));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kern.merge, a, grid);
}

}  // namespace pa
