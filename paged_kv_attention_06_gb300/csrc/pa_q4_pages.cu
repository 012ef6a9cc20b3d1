// Write path and read-back of 4-bit page pools.
//
// Writing: of each group of 32 elements of a new K or V row,
//   y = f16(min(max(x, -448), 448)),  m = min y,  s = f16(fp32(max y - m) / 15),
//   code = the integer nearest to (y - m) / s, ties to even, at most 15 (0 where
//   s is 0);
// a NaN makes its group's m and s NaN. m is one of the values, so the group's least
// is held exactly; s is rounded to the 11 bits that are stored before it is used, so
// that the codes are nearest for the step a reader has.
//
// Reading back: m + s c in fp32 (s c is exact, one rounding in the sum), rounded to
// bf16, into dense rows or into the 128-token pages that the prefill kernels read.
//
// Both are bound by memory. A row of 128 bf16 is 16 lanes of 16 bytes in, 4 bytes of
// codes a lane out (or the other way round), the group's extremes found among 4 lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The code of y = m + t, where the quotient by fp32 arithmetic lies too near a half
// to say on which side it is: in 64 bits, where t and (k + 1/2) s are exact.
__device__ __noinline__ int code_near_half(float y, float m, float s, float q)
{
    const double t = double(y) - double(m);
    const int k = int(floorf(q));
    const double half = (double(k) + 0.5) * double(s);
    return k + (t > half || (t == half && (k & 1)) ? 1 : 0);
}

// One lane's 8 elements of a row (the group's other 24 are in the lanes that differ in
// the low two bits): 8 codes, and the group's step and least value as f16x2.
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t* params)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = __half2float(__float2half_rn(min_nan(max_nan(y[i], -kQ4Max), kQ4Max)));
    float lo = y[0], hi = y[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, y[i]);
        hi = max_nan(hi, y[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
    const float s = __half2float(sh);
    *params = uint32_t(__half_as_ushort(sh)) | uint32_t(__half_as_ushort(__float2half_rn(lo))) << 16;
    // t / s to within 2^-19 of a step, times what a half allows for the rounding of t
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = (y[i] - lo) * inv;
        const float r = rintf(q);
        int c = int(r);
        if (fabsf(q - r) > 0.5f - 0x1p-16f)
            c = code_near_half(y[i], lo, s, q);
        codes |= uint32_t(min(max(c, 0), 15)) << (4 * i);
    }
    return codes;
}

// Lane group of 16 per (request, KV head, token) row, K then V.
__global__ void __launch_bounds__(256) append_q4_kernel(const AppendArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    uint8_t* const kp = reinterpret_cast<uint8_t*>(a.key_pages);
    uint8_t* const vp = reinterpret_cast<uint8_t*>(a.value_pages);
    const int64_t rows = int64_t(a.B) * a.H_kv * a.L_new;
    const int c = threadIdx.x & 15;
    const int64_t step = int64_t(gridDim.x) * (blockDim.x >> 4);
    const int64_t first = int64_t(blockIdx.x) * (blockDim.x >> 4) + (threadIdx.x >> 4);
    // whole warps stay in the loop: the extremes are found by shuffles
    const int64_t rounds = (rows + step - 1) / step;
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t r = first + k * step;
        const bool live = r < rows;
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
        int64_t dst = -1;
        if (live) {
            kx = *reinterpret_cast<const uint4*>(a.key + r * 128 + c * 8);
            vx = *reinterpret_cast<const uint4*>(a.value + r * 128 + c * 8);
            const int64_t bh = udiv64(r, a.L_new);
            const int i = int(r - bh * a.L_new);
            const int b = int(udiv64(bh, a.H_kv));
            const int h = int(bh - int64_t(b) * a.H_kv);
            const int64_t slot = a.slot_mapping[int64_t(b) * a.L_new + i];
            if (slot >= 0) {
                const int64_t page = udiv64(slot, a.ps);
                if (page < a.num_pages)
                    dst = ((page * a.H_kv + h) * a.ps + (slot - page * a.ps)) * kQ4RowBytes;
                else if (c == 0 && h == 0)
                    atomicOr(a.err, PA_DEVERR_SLOT_BIT);
            }
        }
        uint32_t kpar, vpar;
        const uint32_t kc = quantise8(kx, &kpar), vc = quantise8(vx, &vpar);
        if (dst >= 0) {
            *reinterpret_cast<uint32_t*>(kp + dst + c * 4) = kc;
            *reinterpret_cast<uint32_t*>(vp + dst + c * 4) = vc;
            if ((c & 3) == 0) {
                *reinterpret_cast<uint32_t*>(kp + dst + kQ4CodeBytes + c) = kpar;
                *reinterpret_cast<uint32_t*>(vp + dst + kQ4CodeBytes + c) = vpar;
            }
        }
    }
}

// 8 codes and their group's params -> 8 bf16.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t params)
{
    const float s = __half2float(__ushort_as_half(uint16_t(params & 0xffffu)));
    const float m = __half2float(__ushort_as_half(uint16_t(params >> 16)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(fmaf(float((codes >> (8 * i)) & 15u), s, m),
                           fmaf(float((codes >> (8 * i + 4)) & 15u), s, m));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block per (request, KV head, kReadTokens tokens), 16 lanes a row (8 where D is
// 64). bf16 pools (kQ4 false): rows as they are, for pages that the kernels above them
// cannot read by TMA.
constexpr int kReadTokens = 64;

template <bool kQ4, int D>
__global__ void __launch_bounds__(256) read_pages_kernel(const PageReadArgs a)
{
    constexpr int kLanes = D / 8, kRowsAtOnce = 256 / kLanes;
    constexpr int kRowBytes = kQ4 ? kQ4RowBytes : 2 * D;
    grid_dependency_wait();
    grid_launch_dependents();
    const int chunks = a.chunks;
    const int64_t bh = udiv64(blockIdx.x, chunks);
    const int t0 = int(blockIdx.x - bh * chunks) * kReadTokens;
    const int b = int(udiv64(bh, a.H_kv));
    const int h = int(bh - int64_t(b) * a.H_kv);
    const int cap = int(min(int64_t(a.max_pages) * a.ps, int64_t(a.max_len)));
    int n = a.context_lens[b];
    if (n < 0 || n > cap) {
        if (h == 0 && t0 == 0 && threadIdx.x == 0)
            atomicOr(a.err, PA_DEVERR_CONTEXT_LEN_BIT);
        n = n < 0 ? 0 : cap;
    }
    if (a.table_out && h == 0 && threadIdx.x == 0 && t0 % kQ4CopyRows == 0)
        a.table_out[int64_t(b) * a.copy_pages + t0 / kQ4CopyRows] = int32_t(b * a.copy_pages + t0 / kQ4CopyRows);
    if (t0 >= n)
        return;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int c = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    constexpr int kRounds = kReadTokens / kRowsAtOnce;
    uint4 kx[kRounds], vx[kRounds];         // 4-bit rows: x the codes, y the parameters
    bool live[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int t = t0 + kRowsAtOnce * k + row;
        live[k] = t < n;
        kx[k] = vx[k] = make_uint4(0, 0, 0, 0);
        if (live[k]) {
            const int lp = t / a.ps;
            const int phys = bt[lp];
            if (unsigned(phys) >= unsigned(a.num_pages)) {
                if (c == 0 && h == 0)
                    atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
                live[k] = a.table_out != nullptr;      // a copy's row: zeros; a dense row: left
                continue;
            }
            const int64_t src = ((int64_t(phys) * a.H_kv + h) * a.ps + (t - lp * a.ps)) * kRowBytes;
            if constexpr (kQ4) {
                kx[k].x = *reinterpret_cast<const uint32_t*>(a.key_pages + src + c * 4);
                vx[k].x = *reinterpret_cast<const uint32_t*>(a.value_pages + src + c * 4);
                kx[k].y = *reinterpret_cast<const uint32_t*>(a.key_pages + src + kQ4CodeBytes + (c & 12));
                vx[k].y = *reinterpret_cast<const uint32_t*>(a.value_pages + src + kQ4CodeBytes + (c & 12));
            } else {
                kx[k] = *reinterpret_cast<const uint4*>(a.key_pages + src + c * 16);
                vx[k] = *reinterpret_cast<const uint4*>(a.value_pages + src + c * 16);
            }
        }
    }
    // rows from a pointer of their 128-token block: dense rows follow on, copy pages
    // are apart by the other heads' pages
    const int64_t base = int64_t(b) * a.batch_stride + int64_t(h) * a.head_stride + c * 8;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (!live[k])
            continue;
        const int t = t0 + kRowsAtOnce * k + row;
        const int64_t dst = base + int64_t(t / kQ4CopyRows) * a.block_stride + int64_t(t % kQ4CopyRows) * D;
        *reinterpret_cast<uint4*>(a.key_out + dst) = kQ4 ? values8(kx[k].x, kx[k].y) : kx[k];
        *reinterpret_cast<uint4*>(a.value_out + dst) = kQ4 ? values8(vx[k].x, vx[k].y) : vx[k];
    }
}

}  // namespace

cudaError_t launch_append_q4(const AppendArgs& a, cudaStream_t stream)
{
    const int64_t rows = int64_t(a.B) * a.L_new * a.H_kv;
    if (rows == 0)
        return cudaSuccess;
    int64_t blocks = (rows + 15) / 16;
    if (blocks > 65535)
        blocks = 65535;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_q4_kernel, a);
}

cudaError_t launch_read_pages(PageReadArgs a, int kind, int D, cudaStream_t stream)
{
    a.chunks = int32_t((int64_t(a.max_len) + kReadTokens - 1) / kReadTokens);
    const int64_t blocks = int64_t(a.B) * a.H_kv * a.chunks;
    if (blocks <= 0 || blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg,
                              kind == kQ4Pool ? read_pages_kernel<true, 128>
                              : D == 64       ? read_pages_kernel<false, 64>
                                              : read_pages_kernel<false, 128>,
                              a);
}

}  // namespace pa
