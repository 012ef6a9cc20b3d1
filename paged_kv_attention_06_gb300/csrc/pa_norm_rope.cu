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
// operations in between. A row (token, head) is held by D / 8 lanes; in the
// half form a lane holds four elements and their four partners, so the
// rotation needs no exchange and half the angles that eight neighbours would
// (8 bytes a load, each group of lanes still covering whole 128-byte lines). A
// group of lanes takes U heads of one kind of one token: all loads are issued
// before the first is used, and the products of weights and angles are made once
// for the U heads, two elements to an instruction. Measured (one call of a
// replayed graph): 8188 tokens of 32 + 2 x 8 heads of 128, 204.6 MB, 35 us (5.8
// TB/s, of 6.8 for a copy), e4m3 pools 42 us (188.7 MB, 4.5 TB/s: presumably the division
// and the narrow stores of the codes); one token 2.0 us. What is left is the
// latency of a block's loads.
//
// Loads and bf16 stores are marked as streamed (evict first): 39.2 us without. Marking
// one side alone gained nothing when it was measured (38.7 us without, 38.8 with the
// stores' alone, 40 with the loads' alone, 34.7 with both). The attention that follows does not
// pay for it: qkv written, appended and attended to (window 1024), 8188 tokens 178 us
// against 181, 4094 tokens 97 against 98, 1024 tokens 33.4 both.
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// 8188 tokens 35.1 us, e4m3 pools 42.3; 256 threads 35.9 and 48.4, 64 threads 35.3 us.
constexpr int kThreads = 128;

// Four bf16 -> two fp32 pairs, and back.
__device__ __forceinline__ void unpack4(uint2 v, float2* x)
{
    x[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    x[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ uint2 pack4(const float2* x)
{
    return make_uint2(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y));
}
// The e4m3 codes of four quotients x / scale, each rounded to fp32 first. (A product
// with 1 / scale, and the division only where the code could differ, is slower with
// 128 threads a block: 8188 tokens 43.7 us, 42.3 with the division alone.)
__device__ __forceinline__ uint32_t quantise4(const float2* x, float scale)
{
    return f32x2_to_e4m3x2(__fdiv_rn(x[0].x, scale), __fdiv_rn(x[0].y, scale)) |
           (f32x2_to_e4m3x2(__fdiv_rn(x[1].x, scale), __fdiv_rn(x[1].y, scale)) << 16);
}

// One group of D / 8 lanes: up to U neighbouring heads of one kind (queries,
// keys or values) of one token; a.q_groups groups for the queries, a.kv_groups
// each for keys and values.
template <int D, int U, bool kInter, bool kF8>
__global__ void __launch_bounds__(kThreads) norm_rope_append_kernel(const NormRopeArgs a)
{
    constexpr int kLanes = D / 8;
    // The previous kernel in the stream may still write qkv or read the pools.
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t group = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int c = threadIdx.x & (kLanes - 1);
    const int per_token = a.q_groups + 2 * a.kv_groups;
    const int64_t tok_u = udiv64(group, per_token);
    const int j = int(group - tok_u * per_token);
    const int kind = j < a.q_groups ? 0 : j < a.q_groups + a.kv_groups ? 1 : 2;   // q, k, v
    const int h0 = (kind == 0 ? j : j - a.q_groups - (kind == 2 ? a.kv_groups : 0)) * U;
    // Groups past the last token stay for the shuffles and write nothing.
    const bool live = tok_u < int64_t(a.B) * a.L;
    const int heads = live ? min(U, (kind == 0 ? a.H_q : a.H_kv) - h0) : 0;
    const int64_t tok = live ? tok_u : 0;
    const int b = int(udiv64(tok, a.L));
    const int i = int(tok - int64_t(b) * a.L);
    // This lane's two runs of four elements, starting at e0 and e1. Half form:
    // a run and its partners R / 2 further on, or two runs behind R.
    // Interleaved form: eight neighbours.
    const int R = a.rotary_dim;
    const bool turns = kind < 2 && 8 * c < R;
    const bool apart = !kInter && 8 * c < R;
    const int e0 = apart ? 4 * c : 8 * c;
    const int e1 = apart ? 4 * c + R / 2 : 8 * c + 4;

    const uint16_t* src = a.qkv + int64_t(b) * a.batch_stride + int64_t(i) * a.token_stride +
                          ((kind == 0 ? 0 : kind == 1 ? a.H_q : a.H_q + a.H_kv) + h0) * D;
    uint2 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u][0] = raw[u][1] = make_uint2(0, 0);
        if (u < heads) {
            raw[u][0] = __ldcs(reinterpret_cast<const uint2*>(src + u * D + e0));
            raw[u][1] = __ldcs(reinterpret_cast<const uint2*>(src + u * D + e1));
        }
    }
    const int64_t slot = a.slot_mapping[tok];
    // The row is y = inv * (x A + p B), p the partners: with the weights w and
    // the angles, A = w cos and B = +- w' sin, made once for the U heads.
    // Half form: x[0..1] and x[2..3] are partners; interleaved form: the two of
    // each pair.
    float2 A[4], B[4];
    const uint16_t* w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    if (w != nullptr) {
        unpack4(*reinterpret_cast<const uint2*>(w + e0), A);
        unpack4(*reinterpret_cast<const uint2*>(w + e1), A + 2);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            A[k] = make_float2(1.f, 1.f);
    }
    if (R > 0 && kind < 2) {
        int pos = a.positions[tok];
        if (pos < 0 || pos >= a.table_len) {
            if (live && slot >= 0 && c == 0 && j == 0)
                atomicOr(a.err, PA_DEVERR_POSITION_BIT);
            pos = pos < 0 ? 0 : a.table_len - 1;
        }
        if (turns) {
            const float* row = a.cos_sin + int64_t(pos) * R + 4 * c;    // angles 4 c .. 4 c + 3
            const float4 cs = *reinterpret_cast<const float4*>(row);
            const float4 sn = *reinterpret_cast<const float4*>(row + R / 2);
            if constexpr (kInter) {
                const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    B[k] = make_float2(-A[k].y * ss[k], A[k].x * ss[k]);
                    A[k] = make_float2(A[k].x * cc[k], A[k].y * cc[k]);
                }
            } else {
                const float2 cc[2] = {make_float2(cs.x, cs.y), make_float2(cs.z, cs.w)};
                const float2 ss[2] = {make_float2(sn.x, sn.y), make_float2(sn.z, sn.w)};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    B[k] = make_float2(-A[2 + k].x * ss[k].x, -A[2 + k].y * ss[k].y);
                    B[2 + k] = make_float2(A[k].x * ss[k].x, A[k].y * ss[k].y);
                    A[k] = make_float2(A[k].x * cc[k].x, A[k].y * cc[k].y);
                    A[2 + k] = make_float2(A[2 + k].x * cc[k].x, A[2 + k].y * cc[k].y);
                }
            }
        }
    }
    // Where head h0's row goes (elements), and the step from head to head.
    uint16_t* to = a.query;
    int64_t at = ((int64_t(b) * a.H_q + h0) * a.L + i) * D, head_step = int64_t(a.L) * D;
    int stored = heads;
    if (kind > 0) {
        to = kind == 1 ? a.key_pages : a.value_pages;
        head_step = int64_t(D) << a.ps_shift;
        const int64_t page = slot >> a.ps_shift;
        if (slot < 0 || page >= a.num_pages) {
            if (slot >= 0 && live && c == 0 && h0 == 0)
                atomicOr(a.err, PA_DEVERR_SLOT_BIT);
            stored = 0;
        } else {
            at = (((page * a.H_kv + h0) << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * D;
        }
    }
    const bool quantised = kF8 && kind > 0;
    const float scale = kind == 1 ? a.k_scale : a.v_scale;
    const bool normed = __any_sync(0xffffffffu, w != nullptr);

#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 x[4];
        unpack4(raw[u][0], x);
        unpack4(raw[u][1], x + 2);
        float inv = 1.f;
        if (normed) {
            float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
            for (int k = 1; k < 4; ++k)
                s2 = __ffma2_rn(x[k], x[k], s2);
            float sum = s2.x + s2.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (w != nullptr)
                inv = rsqrtf(sum * (1.f / D) + a.eps);
        }
        if (u >= stored)
            continue;
        uint2 out[2] = {raw[u][0], raw[u][1]};       // values of bf16 pools: as they are
        if (kind < 2) {
            const float2 inv2 = make_float2(inv, inv);
            float2 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[k] = __fmul2_rn(x[k], A[k]);
            if (turns) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = __ffma2_rn(kInter ? make_float2(x[k].y, x[k].x) : x[k ^ 2], B[k], y[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = __fmul2_rn(y[k], inv2);
            out[0] = pack4(x);
            out[1] = pack4(x + 2);
        }
        if (quantised) {
            uint8_t* row = reinterpret_cast<uint8_t*>(to) + at + u * head_step;
            *reinterpret_cast<uint32_t*>(row + e0) = quantise4(x, scale);
            *reinterpret_cast<uint32_t*>(row + e1) = quantise4(x + 2, scale);
        } else {
            uint16_t* row = to + at + u * head_step;
            __stcs(reinterpret_cast<uint2*>(row + e0), out[0]);
            __stcs(reinterpret_cast<uint2*>(row + e1), out[1]);
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
    // One head per group while that still leaves the GPU short of threads. Four
    // otherwise: 8188 tokens 35.1 us, 43.3 with two, 37.3 with six, 35.6 with eight.
    const bool few = tokens * H * lanes < int64_t(256) * 1024;
    const int U = few ? 1 : kHeads;
    a.q_groups = (a.H_q + U - 1) / U;
    a.kv_groups = (a.H_kv + U - 1) / U;
    const int64_t blocks = (tokens * (a.q_groups + 2 * a.kv_groups) * lanes + kThreads - 1) / kThreads;
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
