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
// weights. A thread holds one position, so the score rows and the page rows are
// read in whole sectors; the R row states are staged in shared memory.
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) accumulate_weights_kernel(const WeightArgs a)
{
    __shared__ float2 state[kThreads];               // (max, 1 / sum) of up to kThreads rows
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t bh = blockIdx.x / a.chunks;
    const int chunk = int(blockIdx.x - bh * a.chunks);
    const int b = int(bh / a.H_kv), h = int(bh - int64_t(b) * a.H_kv);
    int n = a.context_lens[b];
    const int cap = min(a.max_pages << a.ps_shift, a.score_cap);
    n = n < 0 ? 0 : n > cap ? cap : n;               // recorded by the decode pass
    if (chunk * kThreads >= n)
        return;
    const int pos = chunk * kThreads + int(threadIdx.x);
    const float* s = a.scores + bh * a.R * a.score_stride + pos;
    float w = 0.f;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
        __syncthreads();
        const int rows = min(kThreads, a.R - r0);
        if (int(threadIdx.x) < rows) {
            const float2 st = a.row_state[bh * a.R + r0 + threadIdx.x];
            // a row that sees nothing: every score is -inf and weighs 0
            state[threadIdx.x] = make_float2(st.x == -INFINITY ? 0.f : st.x, st.y > 0.f ? 1.f / st.y : 0.f);
        }
        __syncthreads();
        if (pos < n)
            for (int r = 0; r < rows; ++r)
                w = fmaf(fast_exp2(s[(r0 + r) * a.score_stride] - state[r].x), state[r].y, w);
    }
    if (pos >= n)
        return;
    const int phys = a.block_table[int64_t(b) * a.max_pages + (pos >> a.ps_shift)];
    if (unsigned(phys) >= unsigned(a.num_pages))
        return;                                      // recorded by the decode pass
    float* to = a.weight_pages + ((int64_t(phys) * a.H_kv + h) << a.ps_shift) + (pos & ((1 << a.ps_shift) - 1));
    *to = a.decay != 0.f && pos < n - a.L ? fmaf(a.decay, *to, w) : w;
}

}  // namespace

cudaError_t launch_accumulate_weights(WeightArgs a, cudaStream_t stream)
{
    a.chunks = (a.score_cap + kThreads - 1) / kThreads;
    const int64_t blocks = int64_t(a.B) * a.H_kv * a.chunks;
    if (blocks < 1 || blocks >= (int64_t(1) << 31))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, accumulate_weights_kernel, a);
}

}  // namespace pa
