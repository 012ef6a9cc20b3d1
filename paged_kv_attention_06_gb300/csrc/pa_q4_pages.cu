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
// A row of 128 bf16 is 16 lanes of 16 bytes in, 4 bytes of codes a lane out (or the other
// way round), the group's extremes found among 4 lanes. Measured: 4 x 2047 tokens of 8
// heads written, 44 MB, 14.6 us, and 11.8k read back, 63 MB, 13.8; both calls together 26.8 (4.0
// TB/s, of 6.7 for a copy); 32 tokens written 2.1 and 37.6k of 4 heads read back, 101 MB,
// 20.6, together 23.2; one token 1.9 and 300 rows 3.3, 5.3. What bounds them is the latency
// of one pass of loads a block, and the append's instructions (with quotients near a half
// decided in 64 bits it took 48 us alone; streamed loads or stores change nothing).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

// Minimum and maximum of f16 pairs that keep a NaN.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 widen(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// The code of y where the quotient q by fp32 arithmetic may lie too near a half to say on
// which side it is. With t + e = y - m exactly (t rounded, e what that lost), k = floor(q):
// (k + 1/2) s has 16 bits, so t - (k + 1/2) s is exact near the half, and its sum with e
// has the sign of y - m - (k + 1/2) s.
__device__ __forceinline__ float code_near_half(float y, float m, float s, float q)
{
    const float t = y - m, back = t - y, e = (y - (t - back)) - (m + back);
    const float k = floorf(q);
    const float d = fmaf(-(k + 0.5f), s, t) + e;
    return fminf(d > 0.f || (d == 0.f && (int(k) & 1)) ? k + 1.f : k, 15.f);
}

// One lane's 8 elements of a row (the group's other 24 are in the lanes that differ in
// the low two bits): 8 codes, and the group's step and least value as f16x2.
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t* params)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)      // f16 first: what is past 448 is cut the same way
        y[i] = bf16x2_to_f16x2(w[i]);
    uint32_t lo = min2(min2(y[0], y[1]), min2(y[2], y[3])), hi = max2(max2(y[0], y[1]), max2(y[2], y[3]));
    // (least, negated largest) of the pair, then of the four lanes
    lo = min2(__byte_perm(lo, hi ^ 0x80008000u, 0x5410), __byte_perm(lo, hi ^ 0x80008000u, 0x7632));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1)
        lo = min2(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    float2 ends = widen(lo);
    static_assert(kQ4Max == 448.f, "0x5f00");
    if (fminf(ends.x, ends.y) < -kQ4Max) {               // seldom (NaN: the codes are 0 anyway)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = min2(max2(y[i], 0xdf00df00u), 0x5f005f00u);
        lo = min2(max2(lo, 0xdf00df00u), 0x5f005f00u);
        ends = widen(lo);
    }
    const float m = ends.x;
    // (max - m) / 15, correctly rounded: Markstein's correction of the product with the
    // rounded reciprocal. (No underflow: differences of f16 values are 0 or at least 2^-24.)
    const float range = -ends.y - m, part = 1.f / 15.f;
    const float near = range * part;
    const __half sh = __float2half_rn(fmaf(fmaf(-15.f, near, range), part, near));
    const float s = __half2float(sh);
    *params = uint32_t(__half_as_ushort(sh)) | lo << 16;
    // t / s to within 2^-18 of a step, a quarter of what a half is given for it
    const float inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
    const float2 m2 = make_float2(-m, -m), inv2 = make_float2(inv, inv);
    const float2 round2 = make_float2(12582912.f, 12582912.f);      // 1.5 * 2^23: q + that is rounded to a whole
    const float2 back2 = make_float2(-12582912.f, -12582912.f), minus2 = make_float2(-1.f, -1.f);
    float worst = 0.f;
    float2 sum = make_float2(0.f, 0.f);                  // c0 + 16 c2 + 256 c4 + 4096 c6, and c1 + ...
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 q = __fmul2_rn(__fadd2_rn(widen(y[i]), m2), inv2);
        const float2 r = __fadd2_rn(__fadd2_rn(q, round2), back2);
        const float2 d = __ffma2_rn(r, minus2, q);
        worst = fmaxf(worst, fmaxf(fabsf(d.x), fabsf(d.y)));
        sum = __ffma2_rn(sum, make_float2(16.f, 16.f), r);
    }
    // Near a half (one group in 50: bf16 values are coarse), and where s is so small that
    // its own rounding may put a quotient past 15.
    if (worst > 0.5f - 0x1p-16f || s < 0x1p-14f) {
        sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float2 v = widen(y[i]);
            sum.x = fmaf(sum.x, 16.f, code_near_half(v.x, m, s, (v.x - m) * inv));
            sum.y = fmaf(sum.y, 16.f, code_near_half(v.y, m, s, (v.y - m) * inv));
        }
    }
    // the codes of even elements in bits 0-3, 8-11, ..., of odd ones 4 bits on
    auto spread = [](float c) {
        const uint32_t x = __float_as_uint(c + 8388608.f) & 0xffffu;
        const uint32_t y2 = (x | x << 8) & 0x00ff00ffu;
        return (y2 | y2 << 4) & 0x0f0f0f0fu;
    };
    const uint32_t all = spread(sum.x) | spread(sum.y) << 4;
    return s > 0.f ? all : 0u;                           // one value, or a NaN
}

// Lane group of 16 per (request, KV head, token) row, K then V.
__global__ void __launch_bounds__(256) append_q4_kernel(const AppendArgs a, const FixedDivisor by_L,
                                                        const FixedDivisor by_H)
{
    grid_dependency_wait();
    grid_launch_dependents();
    uint8_t* const kp = reinterpret_cast<uint8_t*>(a.key_pages);
    uint8_t* const vp = reinterpret_cast<uint8_t*>(a.value_pages);
    const int rows = a.B * a.H_kv * a.L_new;
    const int c = threadIdx.x & 15;
    const int shift = __ffs(a.ps) - 1;
    // whole warps stay in the loop: the extremes are found by shuffles
    for (int r0 = int(blockIdx.x) * 16; r0 < rows; r0 += int(gridDim.x) * 16) {
        const int r = r0 + int(threadIdx.x >> 4);
        const bool live = r < rows;
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
        int64_t dst = -1;
        if (live) {
            kx = *reinterpret_cast<const uint4*>(a.key + int64_t(r) * 128 + c * 8);
            vx = *reinterpret_cast<const uint4*>(a.value + int64_t(r) * 128 + c * 8);
            const int bh = by_L.of(r), b = by_H.of(bh), h = bh - b * a.H_kv;
            const int slot = a.slot_mapping[b * a.L_new + (r - bh * a.L_new)];
            if (slot >= 0) {
                const int page = slot >> shift;
                if (page < a.num_pages)
                    dst = ((int64_t(page) * a.H_kv + h) * a.ps + (slot & (a.ps - 1))) * kQ4RowBytes;
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

// 8 codes and their group's params -> 8 bf16 or f16.
template <bool kF16>
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t params)
{
    const float s = __half2float(__ushort_as_half(uint16_t(params & 0xffffu)));
    const float m = __half2float(__ushort_as_half(uint16_t(params >> 16)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                        // 2^23 + c, c, m + s c
        const float2 c = __fadd2_rn(make_float2(__uint_as_float(((codes >> (8 * i)) & 15u) | 0x4b000000u),
                                                __uint_as_float(((codes >> (8 * i + 4)) & 15u) | 0x4b000000u)),
                                    make_float2(-8388608.f, -8388608.f));
        const float2 v = __ffma2_rn(c, make_float2(s, s), make_float2(m, m));
        w[i] = kF16 ? pack_f16x2(v.x, v.y) : pack_bf16x2(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block per (request, KV head, kReadTokens tokens), 16 lanes a row (8 where D is
// 64). bf16 pools (kQ4 false): rows as they are, for pages that the kernels above them
// cannot read by TMA. kF16: the values in f16, whose step is an eighth of bf16's (all
// that a row can hold lies within f16's range).
constexpr int kReadTokens = 128;

template <bool kQ4, int D, bool kF16 = false>
__global__ void __launch_bounds__(256) read_pages_kernel(const PageReadArgs a)
{
    constexpr int kLanes = D / 8, kRowsAtOnce = 256 / kLanes;
    constexpr int kRowBytes = kQ4 ? kQ4RowBytes : 2 * D;
    grid_dependency_wait();
    grid_launch_dependents();
    const int bh = a.by_chunks.of(int(blockIdx.x));
    const int first = (int(blockIdx.x) - bh * a.chunks) * kReadTokens;
    const int b = a.by_H.of(bh), h = bh - b * a.H_kv;
    const int cap = int(min(int64_t(a.max_pages) * a.ps, int64_t(a.max_len)));
    int n = a.context_lens[b];
    if (n < 0 || n > cap) {
        if (h == 0 && first == 0 && threadIdx.x == 0)
            atomicOr(a.err, PA_DEVERR_CONTEXT_LEN_BIT);
        n = n < 0 ? 0 : cap;
    }
    if (a.table_out && h == 0 && threadIdx.x == 0)
        a.table_out[int64_t(b) * a.copy_pages + first / kCopyPageRows] = b * a.copy_pages + first / kCopyPageRows;
    static_assert(kReadTokens == kCopyPageRows, "a block writes one page of a copy");
    if (first >= n)
        return;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int shift = __ffs(a.ps) - 1;
    const int c = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    constexpr int kRounds = kReadTokens / kRowsAtOnce;
    uint4 kx[kRounds], vx[kRounds];         // 4-bit rows: x the codes, y the parameters
    bool live[kRounds];
    int phys[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int t = first + kRowsAtOnce * k + row;
        live[k] = t < n;
        phys[k] = live[k] ? __ldg(bt + (t >> shift)) : 0;
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int t = first + kRowsAtOnce * k + row;
        kx[k] = vx[k] = make_uint4(0, 0, 0, 0);
        if (unsigned(phys[k]) >= unsigned(a.num_pages)) {
            if (c == 0 && h == 0)
                atomicOr(a.err, PA_DEVERR_PAGE_ID_BIT);
            live[k] = a.table_out != nullptr;            // a copy's row: zeros; a dense row: left
        } else if (live[k]) {
            const int64_t src = ((int64_t(phys[k]) * a.H_kv + h) * a.ps + (t & (a.ps - 1))) * kRowBytes;
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
    // (128-token blocks of dense rows follow on, copy pages are apart by the other heads'
    // pages)
    const int64_t base = int64_t(b) * a.batch_stride + int64_t(h) * a.head_stride +
                         int64_t(first / kCopyPageRows) * a.block_stride + c * 8;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (!live[k])
            continue;
        const int64_t dst = base + (kRowsAtOnce * k + row) * D;
        *reinterpret_cast<uint4*>(a.key_out + dst) = kQ4 ? values8<false>(kx[k].x, kx[k].y) : kx[k];
        *reinterpret_cast<uint4*>(a.value_out + dst) = kQ4 ? values8<kF16>(vx[k].x, vx[k].y) : vx[k];
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
    FixedDivisor by_L, by_H;
    by_L.set(a.L_new);
    by_H.set(a.H_kv);
    return cudaLaunchKernelEx(&cfg, append_q4_kernel, a, by_L, by_H);
}

cudaError_t launch_read_pages(PageReadArgs a, int kind, int D, cudaStream_t stream)
{
    a.chunks = int32_t((int64_t(a.max_len) + kReadTokens - 1) / kReadTokens);
    const int64_t blocks = int64_t(a.B) * a.H_kv * a.chunks;
    a.by_chunks.set(a.chunks);
    a.by_H.set(a.H_kv);
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
                              kind == kQ4Pool ? (a.f16_values ? read_pages_kernel<true, 128, true>
                                                              : read_pages_kernel<true, 128>)
                              : D == 64       ? read_pages_kernel<false, 64>
                                              : read_pages_kernel<false, 128>,
                              a);
}

}  // namespace pa
