// Accumulation of attention weights, after a decode pass that kept its scores:
// for every cached position j of a request and KV head,
//
//   w_j = sum over the group's heads and query rows of 2^(s_rj - M_r) / l_r
//   weight[slot of j] = decay * weight[slot of j] + w_j
//
// with (M_r, l_r) the final softmax state of row r, and 0 in the place of the
// old weight for the call's own L newest positions, whose slots are new, and
// for every position when decay is 0 (nothing is read then, so slots need no
// set-up). All in fp32; the rows are added in order.
//
// Bound by memory: 4 R bytes of scores a position (mostly still in L2) and 8 of
// weights. A thread holds four neighbouring positions: 16 bytes of each score
// row, and of the page row where pages hold at least four slots and the pool
// is aligned to 16 bytes (otherwise four single slots). The page id and the old
// weights are requested before the scores. 8 requests of 16k-32k tokens, 32 heads on
// 8: 12 us by itself; in a call whose scores are small it is latency, of which the
// early requests hide a part (32 requests up to 4096 tokens: 24.4 -> 22.9 us a call).
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kEach = 4;                             // positions per thread
constexpr int kSpan = kThreads * kEach;

template <bool kVector>
__global__ void __launch_bounds__(kThreads) accumulate_weights_kernel(const WeightArgs a)
{
    __shared__ float2 state[kThreads];               // (max, 1 / sum) of up to kThreads rows
    grid_launch_dependents();
    // Lengths, tables and weights are inputs of the whole call: complete before
    // the decode pass began, and read (from L2) before this kernel waits for it.
    const int64_t bh = blockIdx.x / a.chunks;
    const int chunk = int(blockIdx.x - bh * a.chunks);
    const int b = int(bh / a.H_kv), h = int(bh - int64_t(b) * a.H_kv);
    int n = __ldcg(a.context_lens + b);
    const int cap = min(a.max_pages << a.ps_shift, a.score_cap);
    n = n < 0 ? 0 : n > cap ? cap : n;               // recorded by the decode pass
    if (chunk * kSpan >= n) {
        grid_dependency_wait();                      // no block of the call ends before its first kernels
        return;
    }
    const int pos = chunk * kSpan + int(threadIdx.x) * kEach;
    const int32_t* bt = a.block_table + int64_t(b) * a.max_pages;
    const int fresh = a.decay != 0.f ? n - a.L : 0;  // positions from here on start at 0
    float* to[kEach];
    float old[kEach] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kVector) {
        to[0] = nullptr;
        if (pos < n) {
            const int phys = __ldcg(bt + (pos >> a.ps_shift));
            if (unsigned(phys) < unsigned(a.num_pages)) {    // otherwise recorded by the decode pass
                to[0] = a.weight_pages + ((int64_t(phys) * a.H_kv + h) << a.ps_shift) +
                        (pos & ((1 << a.ps_shift) - 1));
                if (pos < fresh) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(to[0]));
                    old[0] = v.x;
                    old[1] = v.y;
                    old[2] = v.z;
                    old[3] = v.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            to[u] = nullptr;
            if (pos + u < n) {
                const int phys = __ldcg(bt + ((pos + u) >> a.ps_shift));
                if (unsigned(phys) < unsigned(a.num_pages)) {
                    to[u] = a.weight_pages + ((int64_t(phys) * a.H_kv + h) << a.ps_shift) +
                            ((pos + u) & ((1 << a.ps_shift) - 1));
                    if (pos + u < fresh)
                        old[u] = __ldcg(to[u]);
                }
            }
        }
    }
    // A row of scores is a whole number of 64 positions: 16 bytes at pos < n lie
    // within it.
    const float* s = a.scores + bh * a.R * a.score_stride + pos;
    float w[kEach] = {0.f, 0.f, 0.f, 0.f};
    grid_dependency_wait();
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
        __syncthreads();
        const int rows = min(kThreads, a.R - r0);
        // the first scores come with the states
        constexpr int kAhead = 4;
        float4 v[kAhead];
#pragma unroll
        for (int r = 0; r < kAhead; ++r)
            v[r] = pos < n && r < rows ? __ldcg(reinterpret_cast<const float4*>(s + (r0 + r) * a.score_stride))
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (int(threadIdx.x) < rows) {
            const float2 st = a.row_state[bh * a.R + r0 + threadIdx.x];
            // a row that sees nothing: every score is -inf and weighs 0
            state[threadIdx.x] = make_float2(st.x == -INFINITY ? 0.f : st.x, st.y > 0.f ? 1.f / st.y : 0.f);
        }
        __syncthreads();
        auto add = [&](int r, float4 x) {
            const float2 st = state[r];
            w[0] = fmaf(fast_exp2(x.x - st.x), st.y, w[0]);
            w[1] = fmaf(fast_exp2(x.y - st.x), st.y, w[1]);
            w[2] = fmaf(fast_exp2(x.z - st.x), st.y, w[2]);
            w[3] = fmaf(fast_exp2(x.w - st.x), st.y, w[3]);
        };
#pragma unroll
        for (int r = 0; r < kAhead; ++r)
            if (r < rows)
                add(r, v[r]);
        if (pos < n)
#pragma unroll 4
            for (int r = kAhead; r < rows; ++r)
                add(r, __ldcg(reinterpret_cast<const float4*>(s + (r0 + r) * a.score_stride)));
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u)
        if (pos + u < fresh)
            w[u] = fmaf(a.decay, old[u], w[u]);
    if constexpr (kVector) {
        if (to[0] != nullptr) {
            if (pos + kEach <= n) {
                *reinterpret_cast<float4*>(to[0]) = make_float4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int u = 0; u < kEach; ++u)      // slots behind the context stay
                    if (pos + u < n)
                        to[0][u] = w[u];
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            if (to[u] != nullptr)
                *to[u] = w[u];
    }
}

}  // namespace

cudaError_t launch_accumulate_weights(WeightArgs a, cudaStream_t stream)
{
    a.chunks = (a.score_cap + kSpan - 1) / kSpan;
    const int64_t blocks = int64_t(a.B) * a.H_kv * a.chunks;
    if (blocks < 1 || blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    const bool vector = a.ps_shift >= 2 && (reinterpret_cast<uintptr_t>(a.weight_pages) & 15u) == 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, vector ? accumulate_weights_kernel<true> : accumulate_weights_kernel<false>, a);
}

}  // namespace pa
