// Norms of queries and keys for each head, the position rotation, and the
// write path in one pass: the step between a model's fused QKV projection and
// pa_attention (Reading vLLM's PagedAttention Kernel, 3.2 "Writing into the
// cache": the rows a cache stores are the rotated keys and the values).
//
//   y = x * rsqrt(mean(x^2) + eps) * w        per head row of D (w given)
//   half form:        (y_i, y_{i+R/2}) -> (y_i c - y_{i+R/2} s, y_{i+R/2} c + y_i s)
//   interleaved form: (y_2i, y_{2i+1}) -> the same with pairs of neighbours
//   with c, s = the fp32 table's cos and sin of angle i at the token's
//   position; elements from R on are not rotated. Queries go to [B, H_q, L, D],
//   rotated keys and plain values to the slots of the page pools (bf16, or
//   e4m3 codes).
//
// All arithmetic is fp32; each result is rounded once (bf16, or the e4m3
// code nearest to value / scale).
//
// Bound by memory: every element is read once and written once, ten
// operations in between. A row (token, head) is held by D / 8 lanes, 16 bytes
// each, so loads and stores are whole 32-byte sectors and the mean is a
// shuffle tree; a group of lanes takes U heads of one token, all loads issued
// before the first is used, and the token's angles are read once for the U
// heads. In the half form an element's partner sits R / 16 lanes away: its raw
// bf16 words come by shuffle.
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void unpack8(uint4 v, float* x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = bf16x2_to_f32(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float* x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 quantise8(const float* x, float scale)
{
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c[k] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * k], scale), __fdiv_rn(x[2 * k + 1], scale));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One group of D / 8 lanes: heads j, j + gpt, ... (U of them at most) of one
// token, gpt groups per token.
template <int D, int U, bool kInter, bool kF8>
__global__ void __launch_bounds__(kThreads) norm_rope_append_kernel(const NormRopeArgs a)
{
    constexpr int kLanes = D / 8;
    // The previous kernel in the stream may still write qkv or read the pools.
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t group = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int c = threadIdx.x & (kLanes - 1);
    const int H = a.H_q + 2 * a.H_kv;
    const int64_t tok_u = udiv64(group, a.gpt);
    const int j = int(group - tok_u * a.gpt);
    // Groups past the last token stay for the shuffles and write nothing.
    const bool live = tok_u < int64_t(a.B) * a.L;
    const int64_t tok = live ? tok_u : 0;
    const int b = int(udiv64(tok, a.L));
    const int i = int(tok - int64_t(b) * a.L);
    const uint16_t* src = a.qkv + int64_t(b) * a.batch_stride + int64_t(i) * a.token_stride + c * 8;

    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = j + u * a.gpt;
        raw[u] = live && h < H ? *reinterpret_cast<const uint4*>(src + int64_t(h) * D)
                               : make_uint4(0, 0, 0, 0);
    }
    const int64_t slot = a.slot_mapping[tok];

    // This lane's 8 angles: elements [8 c, 8 c + 8) of the row.
    float cs[8], sn[8];
    const int R = a.rotary_dim;
    const bool turns = 8 * c < R;
    const int half_lanes = R / 16;                       // lanes of half a rotation (half form)
    const bool upper = !kInter && c >= half_lanes;       // holds the second elements of its pairs
    if (R > 0) {
        int pos = a.positions[tok];
        if (pos < 0 || pos >= a.table_len) {
            if (live && slot >= 0 && c == 0 && j == 0)
                atomicOr(a.err, PA_DEVERR_POSITION_BIT);
            pos = pos < 0 ? 0 : a.table_len - 1;
        }
        if (turns) {
            const float* row = a.cos_sin + int64_t(pos) * R;
            if constexpr (kInter) {                      // angles 4 c .. 4 c + 3
                const float4 p = *reinterpret_cast<const float4*>(row + 4 * c);
                const float4 q = *reinterpret_cast<const float4*>(row + R / 2 + 4 * c);
                cs[0] = p.x; cs[1] = p.y; cs[2] = p.z; cs[3] = p.w;
                sn[0] = q.x; sn[1] = q.y; sn[2] = q.z; sn[3] = q.w;
            } else {
                const float* at = row + 8 * (upper ? c - half_lanes : c);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 p = *reinterpret_cast<const float4*>(at + 4 * k);
                    const float4 q = *reinterpret_cast<const float4*>(at + R / 2 + 4 * k);
                    cs[4 * k] = p.x; cs[4 * k + 1] = p.y; cs[4 * k + 2] = p.z; cs[4 * k + 3] = p.w;
                    sn[4 * k] = q.x; sn[4 * k + 1] = q.y; sn[4 * k + 2] = q.z; sn[4 * k + 3] = q.w;
                }
            }
        }
    }
    // The slot's row offset in the pools (element of head 0), or -1.
    int64_t dst = -1;
    if (live && slot >= 0) {
        const int64_t page = slot >> a.ps_shift;
        if (page >= a.num_pages) {
            if (c == 0 && j == 0)
                atomicOr(a.err, PA_DEVERR_SLOT_BIT);
        } else {
            dst = ((page * a.H_kv << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * D + c * 8;
        }
    }
    const int partner = !turns ? c : upper ? c - half_lanes : c + half_lanes;   // half form

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = j + u * a.gpt;
        const int kind = h < a.H_q ? 0 : h < a.H_q + a.H_kv ? 1 : 2;   // q, k, v
        float x[8];
        unpack8(raw[u], x);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum = fmaf(x[k], x[k], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        uint4 other = make_uint4(0, 0, 0, 0);
        if constexpr (!kInter) {
            other.x = __shfl_sync(0xffffffffu, raw[u].x, partner, kLanes);
            other.y = __shfl_sync(0xffffffffu, raw[u].y, partner, kLanes);
            other.z = __shfl_sync(0xffffffffu, raw[u].z, partner, kLanes);
            other.w = __shfl_sync(0xffffffffu, raw[u].w, partner, kLanes);
        }
        if (!live || h >= H)
            continue;
        if (kind < 2) {
            const uint16_t* w = kind == 0 ? a.q_weight : a.k_weight;
            float y[8];                                  // the partners, normed
            if constexpr (!kInter)
                unpack8(other, y);
            if (w != nullptr) {
                const float inv = rsqrtf(sum * (1.f / D) + a.eps);
                float wx[8];
                unpack8(*reinterpret_cast<const uint4*>(w + 8 * c), wx);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = x[k] * inv * wx[k];
                if constexpr (!kInter) {
                    unpack8(*reinterpret_cast<const uint4*>(w + 8 * partner), wx);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        y[k] = y[k] * inv * wx[k];
                }
            }
            if (turns) {
                if constexpr (kInter) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p = x[2 * k], q = x[2 * k + 1];
                        x[2 * k] = p * cs[k] - q * sn[k];
                        x[2 * k + 1] = q * cs[k] + p * sn[k];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        x[k] = upper ? x[k] * cs[k] + y[k] * sn[k] : x[k] * cs[k] - y[k] * sn[k];
                }
            }
        }
        if (kind == 0) {
            uint16_t* q = a.query + ((int64_t(b) * a.H_q + h) * a.L + i) * D + c * 8;
            *reinterpret_cast<uint4*>(q) = pack8(x);
        } else if (dst >= 0) {
            const int hk = h - a.H_q - (kind == 2 ? a.H_kv : 0);
            const int64_t at = dst + (int64_t(hk) << a.ps_shift) * D;
            if constexpr (kF8) {
                uint8_t* pool = reinterpret_cast<uint8_t*>(kind == 1 ? a.key_pages : a.value_pages);
                *reinterpret_cast<uint2*>(pool + at) = quantise8(x, kind == 1 ? a.k_scale : a.v_scale);
            } else {
                uint16_t* pool = kind == 1 ? a.key_pages : a.value_pages;
                *reinterpret_cast<uint4*>(pool + at) = kind == 2 ? raw[u] : pack8(x);
            }
        }
    }
}

template <int D, int U>
const void* kernel_for(bool inter, bool fp8)
{
    if constexpr (D == 128) {
        if (fp8)
            return inter ? reinterpret_cast<const void*>(norm_rope_append_kernel<D, U, true, true>)
                         : reinterpret_cast<const void*>(norm_rope_append_kernel<D, U, false, true>);
    }
    return inter ? reinterpret_cast<const void*>(norm_rope_append_kernel<D, U, true, false>)
                 : reinterpret_cast<const void*>(norm_rope_append_kernel<D, U, false, false>);
}

}  // namespace

cudaError_t launch_norm_rope_append(NormRopeArgs a, cudaStream_t stream)
{
    constexpr int kHeads = 4;
    const int H = a.H_q + 2 * a.H_kv;
    const int64_t tokens = int64_t(a.B) * a.L;
    const int lanes = a.D / 8;
    // One head per group while that still leaves the GPU short of threads.
    const bool few = tokens * H * lanes < int64_t(256) * 1024;
    const int U = few ? 1 : kHeads;
    a.gpt = (H + U - 1) / U;
    const int64_t blocks = (tokens * a.gpt * lanes + kThreads - 1) / kThreads;
    if (blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    const void* fn = a.D == 64 ? (few ? kernel_for<64, 1>(a.interleaved, a.fp8) : kernel_for<64, kHeads>(a.interleaved, a.fp8))
                               : (few ? kernel_for<128, 1>(a.interleaved, a.fp8) : kernel_for<128, kHeads>(a.interleaved, a.fp8));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
