/*
 * pagedattn: paged K/V attention for NVIDIA GB300 (sm_103a).
 *
 * A C ABI over hand-written CUDA kernels. Query heads attend over a per-layer
 * pool of fixed-size K/V pages through a per-request block table, without
 * gathering a dense K/V tensor first.
 *
 * Conventions shared by every call:
 *   - All tensors are raw DEVICE pointers to contiguous row-major buffers
 *     owned by the caller. bf16 values are passed as their 16-bit patterns.
 *   - Layouts (Week 3 Day 4: Direct Paged Attention, "The Paged Attention
 *     API" and "How This Maps to tiny-llm"; Tutorial 13: Paged Attention and
 *     Memory Management, section 6 "Paged Attention Metadata"):
 *       query        [B, H_q, L, D]            bf16
 *       out          [B, H_q, L, D]            bf16
 *       key_pages    [P, H_kv, page_size, D]   bf16 (one pool per layer)
 *       value_pages  [P, H_kv, page_size, D]   bf16
 *       block_table  [B, max_pages]            int32, physical page ids
 *       context_lens [B]                       int32, valid tokens per request
 *     Logical position j of request b is slot j % page_size of physical page
 *     block_table[b, j / page_size] (Week 3 Day 4, "Why block_table
 *     Matters"). Entries past ceil(context_lens[b] / page_size) are never
 *     read and may hold anything.
 *   - GQA: query head h_q reads KV head h_q / (H_q / H_kv).
 *   - Causal mask: query row i of request b sits at absolute position
 *     context_lens[b] - L + i (the rows are the newest L positions) and sees
 *     keys 0..that position. With causal = 0 every row sees all
 *     context_lens[b] keys. A row that sees no key returns zeros.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). Every call is asynchronous on it; nothing synchronises except
 *     pa_get_device_error.
 *   - Errors: a call that returns anything but PA_OK launched nothing and
 *     touched no buffer. Per-request values that live on the device
 *     (block_table entries, context_lens, slot_mapping) cannot be checked on
 *     the host; the kernels check them, never access memory outside the
 *     buffers for a bad value, and record it in a device error word that
 *     pa_get_device_error reads.
 *   - The library allocates no device memory on any call.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,    /* null pointer, bad size, bad scale, misalignment */
    PA_ERR_UNSUPPORTED = 2,    /* D not 64/128, H_q % H_kv != 0, page_size not a
                                  power of two in 1..256, shapes beyond limits */
    PA_ERR_WORKSPACE = 3,      /* workspace missing or smaller than required    */
    PA_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed          */
    PA_ERR_DEVICE_BOUNDS = 5,  /* a kernel met an out-of-range page id, slot or
                                  context length (from pa_get_device_error)     */
    PA_ERR_DEVICE_TIMEOUT = 6, /* a kernel's bounded wait on its own copies ran
                                  out (from pa_get_device_error)                */
    PA_ERR_NO_PAGES = 7        /* pa_kv_cache: the page pool or a block-table row
                                  is full; nothing was changed                  */
} pa_status;

/* Bits of the device error word reported by pa_get_device_error. */
#define PA_DEVERR_PAGE_ID      0x1u  /* block_table entry outside [0, P)           */
#define PA_DEVERR_SLOT         0x2u  /* slot_mapping entry >= P * page_size         */
#define PA_DEVERR_CONTEXT_LEN  0x4u  /* context_lens entry < 0 or > max_pages*ps    */
#define PA_DEVERR_TIMEOUT      0x8u  /* pipeline wait gave up                       */
#define PA_DEVERR_POSITION     0x10u /* positions entry outside [0, table_len)      */
#define PA_DEVERR_PREFIX       0x20u /* prefix_starts that do not ascend in the batch */

/* Problem sizes shared by every call. */
typedef struct pa_shape {
    int32_t batch;         /* B: requests                                       */
    int32_t num_q_heads;   /* H_q (unused by pa_append_kv)                      */
    int32_t num_kv_heads;  /* H_kv, must divide H_q                             */
    int32_t head_dim;      /* D: 64 or 128                                      */
    int32_t q_len;         /* L: query rows per request; for pa_append_kv the
                              number of new tokens per request (L_new)          */
    int32_t num_pages;     /* P: pages in the pool                              */
    int32_t max_pages;     /* row length (stride) of block_table                */
} pa_shape;

/*
 * Write path: scatter new K/V rows into the page pool by slot_mapping.
 * (Reading vLLM's PagedAttention Kernel, 3.2 "Writing into the cache":
 * the flat slot of a token is physical_block * page_size + offset.)
 *
 *   key, value      [B, H_kv, L_new, D] bf16, 16-byte aligned
 *   key_pages, value_pages  [P, H_kv, page_size, D] bf16, modified in place
 *   slot_mapping    [B, L_new] int32. slot < 0: no token (padding), skipped.
 *                   slot >= P * page_size: skipped, PA_DEVERR_SLOT recorded.
 *                   Two tokens with the same slot: undefined which one lands.
 *   shape.q_len = L_new; shape.num_q_heads and shape.max_pages are unused.
 * The copy is bit-exact.
 */
pa_status pa_append_kv(const void *key, const void *value, void *key_pages,
                       void *value_pages, const int32_t *slot_mapping,
                       int32_t page_size, pa_shape shape, void *stream);

/*
 * Bytes of scratch workspace pa_decode needs for `shape` on the CURRENT
 * device (it depends on the device's SM count). 0 on invalid shapes.
 * It holds one partial (max, sum, output) state per block for every segment
 * (request x KV head x tile of 16 query rows; at most 65536 segments) that
 * straddles blocks; its contents on entry do not matter.
 */
size_t pa_decode_workspace_bytes(pa_shape shape);

/*
 * Decode attention: split-KV over the cached context (Week 3 Day 4,
 * "Choose a Schedule for Each Query Shape" and "Task 2": partition the
 * context across parallel workers and merge their partial (max, sum,
 * output) states; Reading vLLM's PagedAttention Kernel, 3.3: partitions
 * computed in parallel and combined afterwards). Any L >= 1 is computed
 * correctly; the schedule is built for small L (one-token decode).
 *
 *   scale            > 0 and finite (the Python binding maps None to 1/sqrt(D))
 *   max_context_len  an upper bound of context_lens used only to size the
 *                    grid (0 = unknown); larger entries are still correct.
 *   workspace        device scratch of at least pa_decode_workspace_bytes
 *                    bytes, 16-byte aligned; any contents. Calls that share a
 *                    workspace must not overlap on the GPU.
 * The work is two kernels on `stream`: the split-KV pass and a small merge
 * pass, chained by programmatic dependent launch (each waits for the kernel
 * before it in the stream before touching any data).
 */
pa_status pa_decode(const void *query, const void *key_pages,
                    const void *value_pages, const int32_t *block_table,
                    const int32_t *context_lens, int32_t page_size, float scale,
                    int causal, void *out, pa_shape shape,
                    int32_t max_context_len, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * pa_decode without a caller-provided workspace. (The pages have no
 * counterpart: this entry point exists for callers of this library that
 * cannot allocate device memory, e.g. a host program embedded in another
 * runtime that owns every device allocation and only hands out the input and
 * output pointers, or a serving loop where cudaMalloc/cudaFree are off limits
 * because they can synchronise the device mid-flight.)
 *
 * Same arguments, checks and result as pa_decode, minus the workspace: the
 * scratch is a 32 MiB array inside the library's device image, held by every
 * GPU that loads this part of the library until the process exits. The call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 *   - The first call on a device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *   - Shapes whose scratch (pa_decode_workspace_bytes) exceeds 32 MiB are
 *     rejected with PA_ERR_WORKSPACE before anything is launched.
 *   - Every call on a device shares the one array, which keeps the previous
 *     call's contents (the decode needs nothing in it to start at zero).
 *     Calls that overlap on the GPU (other streams, other host threads) race
 *     on the array: order them.
 *   - The array's device address is cached per device for the life of the
 *     process. cudaDeviceReset (or any reset of the device's primary
 *     context) ends the context it was looked up in, and with it the cached
 *     address (and that of the library's device error word): do not call
 *     this library on a device after resetting it in the same process.
 */
pa_status pa_decode_noalloc(const void *query, const void *key_pages,
                            const void *value_pages, const int32_t *block_table,
                            const int32_t *context_lens, int32_t page_size,
                            float scale, int causal, void *out, pa_shape shape,
                            int32_t max_context_len, void *stream);

/*
 * Dense baseline, first step (Week 3 Day 4, "Measure the Direct Page Walk":
 * the dense path gathers each request's cached K/V into contiguous memory
 * before attending; the direct page walk does without this copy). Copies,
 * for every request b, KV head h and position t < context_lens[b], the row
 * pages[block_table[b][t / page_size]][h][t % page_size][:] of key_pages and
 * value_pages into key_dense[b][h][t][:] and value_dense[b][h][t][:].
 *   key_dense, value_dense  device, [B, H_kv, dense_len, D] bf16, 16-byte
 *                           aligned, owned by the caller; rows at or past a
 *                           request's context are not written.
 *   shape                   batch, num_kv_heads, head_dim, num_pages,
 *                           max_pages are used.
 * A block-table entry outside the pool skips its rows and records
 * PA_DEVERR_PAGE_ID; a context longer than dense_len or the block table
 * records PA_DEVERR_CONTEXT_LEN and is cut to fit. Bit copy, one kernel on
 * `stream` (programmatic dependent launch, like pa_append_kv).
 */
pa_status pa_gather_kv(const void *key_pages, const void *value_pages,
                       const int32_t *block_table, const int32_t *context_lens,
                       int32_t page_size, pa_shape shape, int32_t dense_len,
                       void *key_dense, void *value_dense, void *stream);

/*
 * Dense baseline, second step: decode attention over dense K/V buffers
 * [B, H_kv, dense_len, D] (as pa_gather_kv writes them), with the same
 * split-KV kernel, arithmetic and workspace as pa_decode; request b's keys
 * are rows 0 .. context_lens[b] - 1 of its block, no block table is read.
 * On the same K/V values the result is bit-identical to pa_decode's.
 *   dense_len  a multiple of 64, >= every context length (a longer context
 *              records PA_DEVERR_CONTEXT_LEN and is cut to dense_len).
 *   shape      num_pages and max_pages are ignored.
 *   workspace  as for pa_decode (pa_decode_workspace_bytes of the shape).
 */
pa_status pa_decode_dense(const void *query, const void *key_dense,
                          const void *value_dense, const int32_t *context_lens,
                          int32_t dense_len, float scale, int causal, void *out,
                          pa_shape shape, int32_t max_context_len, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * Prefill attention: query rows in tiles, every K/V tile resolved through
 * block_table (Week 3 Day 4, "Task 2", the long-query page-walking
 * schedule), causal by default with the bottom-right offset above. Needs no
 * workspace. Tensor-core kernels (tcgen05, TMEM) for head_dim 128 or 64 and
 * every page size. A KV group of one query head computes that head in both
 * halves of a two-head block. Pages of fewer than 8 tokens are copied into
 * shared memory row by row instead of one TMA box per page.
 */
pa_status pa_prefill(const void *query, const void *key_pages,
                     const void *value_pages, const int32_t *block_table,
                     const int32_t *context_lens, int32_t page_size, float scale,
                     int causal, void *out, pa_shape shape, void *stream);

/*
 * FP8 page pools (Reading vLLM's PagedAttention Kernel, section 3.2: the
 * write path takes the cache dtype and per-tensor k_scale / v_scale). A pool
 * holds e4m3 codes (1 byte per element: sign, 4 exponent bits with bias 7,
 * 3 mantissa bits, largest finite 448), [num_pages, num_kv_heads, page_size,
 * head_dim] like the bf16 pools; a code c stands for value(c) * scale.
 * head_dim 128 only.
 */

/*
 * pa_append_kv for e4m3 pools: every element of the new rows (bf16) is
 * stored as the e4m3 code nearest to fp32(x) / scale (the quotient rounded to
 * fp32 first; ties to the even code; magnitudes past 448 saturate to 448; a
 * NaN gives a NaN code). k_scale and v_scale must be finite and > 0. Same
 * slots, checks and error reporting as pa_append_kv.
 */
pa_status pa_append_kv_fp8(const void *key, const void *value, void *key_pages,
                           void *value_pages, const int32_t *slot_mapping, int32_t page_size,
                           float k_scale, float v_scale, pa_shape shape, void *stream);

/*
 * From a fused QKV projection to the cache in one pass: the norm of every
 * query and key head row, the position rotation, and the write path (Reading
 * vLLM's PagedAttention Kernel, 3.2: the cache holds rotated keys and plain
 * values). The queries it writes are pa_attention's, the K/V rows those of
 * pa_append_kv.
 *   qkv          bf16. Token (b, i) is a row of (H_q + 2 H_kv) D elements at
 *                element b * qkv_batch_stride + i * qkv_token_stride: H_q query
 *                heads, then H_kv key heads, then H_kv value heads. 16-byte
 *                aligned, strides in elements, multiples of 8, at least a row.
 *   q_weight, k_weight   [D] bf16, 16-byte aligned: x * rsqrt(mean(x^2) + eps)
 *                * weight for each head row; NULL: no norm of queries / keys.
 *   cos_sin      [table_len, rotary_dim] fp32, 16-byte aligned: for each
 *                position the cosines of the rotary_dim / 2 angles, then their
 *                sines (made once, in as many bits as far positions need).
 *   rotary_dim   R, a multiple of 16 up to D: the first R elements of a head
 *                row are rotated, in pairs (i, i + R/2), or (2i, 2i + 1) when
 *                interleaved. 0: no rotation (cos_sin, positions unused).
 *   positions    [B, L] int32, each token's row of cos_sin. A token's position
 *                and its slot are independent (an evicted cache is shorter
 *                than the text). An entry outside [0, table_len) records
 *                PA_DEVERR_POSITION and is moved to the nearer end.
 *   query        [B, H_q, L, D] bf16 out, must not overlap qkv. Row i is token
 *                i's: for pa_attention, whose rows are the newest, a request
 *                with fewer than L tokens has its padding tokens first.
 *   slot_mapping [B, L] int32 as for pa_append_kv. A token with slot < 0 is
 *                padding: no K/V is written, and its query row holds the
 *                result for the position clamped into the table (not recorded).
 *   shape        num_q_heads, num_kv_heads, head_dim, q_len = L, num_pages,
 *                batch; max_pages is unused.
 * fp32 arithmetic; queries and bf16 rows are rounded once, e4m3 rows (the
 * _fp8 form, head_dim 128) are the codes pa_append_kv_fp8 gives for the
 * unrounded values. Values are copied bit for bit into bf16 pools.
 */
pa_status pa_qk_norm_rope_append(const void *qkv, int64_t qkv_batch_stride,
                                 int64_t qkv_token_stride, const void *q_weight,
                                 const void *k_weight, float eps, const float *cos_sin,
                                 int32_t rotary_dim, int32_t table_len, int interleaved,
                                 const int32_t *positions, void *query, void *key_pages,
                                 void *value_pages, const int32_t *slot_mapping,
                                 int32_t page_size, pa_shape shape, void *stream);
pa_status pa_qk_norm_rope_append_fp8(const void *qkv, int64_t qkv_batch_stride,
                                     int64_t qkv_token_stride, const void *q_weight,
                                     const void *k_weight, float eps, const float *cos_sin,
                                     int32_t rotary_dim, int32_t table_len, int interleaved,
                                     const int32_t *positions, void *query, void *key_pages,
                                     void *value_pages, const int32_t *slot_mapping,
                                     int32_t page_size, float k_scale, float v_scale,
                                     pa_shape shape, void *stream);

/*
 * pa_decode over e4m3 pools: the same split-KV schedule, arguments,
 * workspace (pa_decode_workspace_bytes) and result as pa_decode, with every
 * K element value(code) * k_scale and every V element value(code) * v_scale.
 * The kernel reads the codes straight from the pages (half the bytes of the
 * bf16 pools) and multiplies on the tensor cores in f16, into which e4m3
 * values convert exactly; the query is taken in f16 too, so its elements
 * must have magnitudes within f16's range (below 65504; below 2^-14 they keep
 * fewer bits). A NaN code in a visible slot gives NaN; slots past a
 * request's context are never read. Any query length;
 * for prefill chunks pa_prefill_fp8 is the faster call.
 */
pa_status pa_decode_fp8(const void *query, const void *key_pages, const void *value_pages,
                        const int32_t *block_table, const int32_t *context_lens, int32_t page_size,
                        float scale, float k_scale, float v_scale, int causal, void *out,
                        pa_shape shape, int32_t max_context_len, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace pa_prefill_fp8 needs for `shape` (head_dim 128)
 * with contexts of at most max_context_len tokens, on the CURRENT device; 0
 * on invalid shapes. It holds bf16 copies of K and V in pages of 128 tokens
 * (batch * ceil(max_context_len / 128) pages of num_kv_heads * 128 * 128
 * elements each, 64 KiB per page and KV head for K and V together), their
 * page table, and the split prefill's workspace when pa_prefill_fp8 takes
 * that kernel for the shape, or the pairs kernel's tail pieces' (the same
 * rules as pa_attention's prefill route).
 */
size_t pa_prefill_fp8_workspace_bytes(pa_shape shape, int32_t max_context_len);

/*
 * Prefill attention over e4m3 pools (the pools of pa_append_kv_fp8): the
 * result of pa_decode_fp8 (every K element value(code) * k_scale, every V
 * element value(code) * v_scale, bottom-right causal mask when `causal`) on
 * the tensor-core prefill kernels. Two kernels on `stream`:
 *   1. the K/V tokens each request can see are copied into bf16 pages of
 *      128 tokens in the workspace, each code converted to its exact value
 *      (e4m3 values are bf16 values; a NaN code stays NaN);
 *   2. the kernels of pa_attention's prefill route (pa_prefill's, with tail
 *      pieces at 1.5 to 2 items per SM, or pa_prefill_split's below 1.5)
 *      attend over the copies, with scale * k_scale as the softmax scale and
 *      the output multiplied by v_scale, so the scaled values are never
 *      rounded.
 * Arguments as pa_decode_fp8. max_context_len bounds context_lens and sizes
 * the copy; a longer entry records PA_DEVERR_CONTEXT_LEN and is cut to
 * ceil(max_context_len / 128) * 128 tokens. workspace: at least
 * pa_prefill_fp8_workspace_bytes(shape, max_context_len) bytes, 256-byte
 * aligned, any contents; calls sharing one must not overlap on the GPU.
 * head_dim 128 only (PA_ERR_UNSUPPORTED otherwise); k_scale and v_scale
 * finite and > 0 (PA_ERR_INVALID_ARG).
 */
pa_status pa_prefill_fp8(const void *query, const void *key_pages, const void *value_pages,
                         const int32_t *block_table, const int32_t *context_lens,
                         int32_t page_size, float scale, float k_scale, float v_scale, int causal,
                         void *out, pa_shape shape, int32_t max_context_len, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * The dispatch of pa_attention for e4m3 pools: pa_decode_fp8 for query rows
 * L <= 8 (the page's rule: the e4m3 decode reads K/V once per 16-row tile of
 * a KV group), pa_prefill_fp8 otherwise, with the same arguments. The workspace is the one that call takes, at
 * least pa_attention_fp8_workspace_bytes(shape, max_context_len) bytes,
 * 256-byte aligned (0 bytes: invalid shape or head_dim other than 128).
 */
size_t pa_attention_fp8_workspace_bytes(pa_shape shape, int32_t max_context_len);
pa_status pa_attention_fp8(const void *query, const void *key_pages, const void *value_pages,
                           const int32_t *block_table, const int32_t *context_lens,
                           int32_t page_size, float scale, float k_scale, float v_scale,
                           int causal, void *out, pa_shape shape, int32_t max_context_len,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace pa_prefill_split needs for `shape` and
 * page_size on the CURRENT device, or 0 when the shape takes a prefill
 * kernel that needs none (head_dim 64, page_size < 8, one query head per
 * KV group). The size depends only on the device's SM count (about 130 KiB
 * per SM), not on the batch.
 */
size_t pa_prefill_workspace_bytes(pa_shape shape, int32_t page_size);

/*
 * Prefill attention with the same arguments, result and checks as
 * pa_prefill, on a kernel that balances the work over the GPU: the K/V
 * tiles of every (request, pair of query heads of one KV group, tile of 128
 * query rows; with an odd group size the last pair of each group holds its
 * last head twice and writes it once) form one stream, cut into equal
 * ranges for a persistent grid
 * of one block per SM (the split-KV idea of Week 3 Day 4, "Choose a
 * Schedule for Each Query Shape", applied to the long-query schedule). An
 * item cut by range boundaries is finished by the block holding its first
 * tiles, which merges the partial softmax states its later pieces (done
 * first by the following blocks) left in the workspace. The launch is
 * cooperative (all blocks resident); where the device cannot hold every
 * block at once, the call runs pa_prefill's kernels instead.
 *   workspace        device memory of at least pa_prefill_workspace_bytes,
 *                    256-byte aligned, any contents (nothing needs clearing;
 *                    each launch tags its counters with its own stamp).
 *                    Calls that share a workspace must not overlap on the GPU.
 * Shapes for which pa_prefill_workspace_bytes is 0 run pa_prefill (the
 * workspace is then not touched). PA_ERR_WORKSPACE when the workspace is
 * missing, too small or misaligned. The output is the same softmax as
 * pa_prefill's up to rounding (the pieces' states are combined in fp32).
 */
pa_status pa_prefill_split(const void *query, const void *key_pages,
                           const void *value_pages, const int32_t *block_table,
                           const int32_t *context_lens, int32_t page_size, float scale,
                           int causal, void *out, pa_shape shape, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * Route chosen by pa_attention for these sizes: 0 = decode, 1 = prefill.
 * The rule sits at this boundary (Week 3 Day 4, "Choose a Schedule for Each
 * Query Shape": short queries take the vector decode schedule, long ones the
 * page-walking prefill; no dense fallback). The thresholds are this
 * library's, set by timing both kernels on GB300 (the page's own rule,
 * L <= 8, was set on other hardware): decode for L <= 24, and for L <= 32
 * when max_context_len >= 3072; prefill otherwise. Returns -1 on invalid
 * shapes.
 */
int32_t pa_attention_route(pa_shape shape, int32_t max_context_len);

/*
 * Dispatching entry point: runs pa_decode or pa_prefill as
 * pa_attention_route says, with the same arguments. The workspace is
 * required only when the route is decode. On the prefill route, given a
 * workspace of at least pa_prefill_workspace_bytes (256-byte aligned), it
 * runs pa_prefill_split when the shape has fewer than 1.5 (request, head
 * pair, 128-row query tile) items per SM, where whole blocks would leave
 * SMs idle; otherwise pa_prefill's kernel, and with one to two items per SM
 * (head_dim 128) that kernel balances the blocks through the workspace: a
 * block holding two items hands the last K/V tiles of its second item to a
 * block holding one, which runs them first and leaves their softmax state
 * (O / l in bf16, the maximum and the sum in fp32); the first block merges it
 * at its end. No block waits for another: the side that arrives second merges
 * (normally the first block), and both sides merge with the same arithmetic,
 * so the bits do not depend on the order. The output is the same softmax up
 * to rounding. With NULL or a smaller workspace: pa_prefill as it is.
 */
pa_status pa_attention(const void *query, const void *key_pages,
                       const void *value_pages, const int32_t *block_table,
                       const int32_t *context_lens, int32_t page_size,
                       float scale, int causal, void *out, pa_shape shape,
                       int32_t max_context_len, void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * pa_decode with a sliding window and a few first tokens that stay visible:
 * query row i of a request, at position p = context_lens - L + i, sees the
 * keys j <= p with j > p - window or j < sinks (always causal). A row at a
 * negative position returns zeros.
 *   window >= 1, sinks >= 0.
 * Only the pages that hold a key some row sees are touched: block_table
 * entries of the others are not read and may hold anything, so a cache can give
 * back the pages between the sinks and the window. Within the pages that are
 * read, slots that no row of the call sees may hold any bytes; a slot that one
 * row sees and another does not has to hold numbers (0 * NaN in P . V).
 * workspace: pa_decode_window_workspace_bytes(shape) bytes (0: invalid shape),
 * 16-byte aligned, any contents; calls that share one must not overlap on the
 * GPU. Other arguments and the errors as for pa_decode / pa_decode_fp8.
 * Up to 16 rows per request and KV head (G * L) take kernels of their own; more
 * take pa_decode's. Two kernels on `stream`. The e4m3 form takes the query and the
 * softmax weights in f16, as pa_decode_fp8 (query elements below 65504 in
 * magnitude; below 2^-14 they keep fewer bits).
 */
size_t pa_decode_window_workspace_bytes(pa_shape shape);
pa_status pa_decode_window(const void *query, const void *key_pages, const void *value_pages,
                           const int32_t *block_table, const int32_t *context_lens,
                           int32_t page_size, float scale, int32_t window, int32_t sinks,
                           void *out, pa_shape shape, int32_t max_context_len, void *workspace,
                           size_t workspace_bytes, void *stream);
pa_status pa_decode_window_fp8(const void *query, const void *key_pages, const void *value_pages,
                               const int32_t *block_table, const int32_t *context_lens,
                               int32_t page_size, float scale, float k_scale, float v_scale,
                               int32_t window, int32_t sinks, void *out, pa_shape shape,
                               int32_t max_context_len, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * Prefill with a sliding window and first tokens that stay visible: the rows,
 * masks and page rules of pa_decode_window on pa_prefill's tensor-core kernel
 * (two query heads of a KV group per block), each tile of 128 query rows
 * visiting the tiles of the sinks and those its rows see through the window.
 * Needs no workspace.
 */
pa_status pa_prefill_window(const void *query, const void *key_pages, const void *value_pages,
                            const int32_t *block_table, const int32_t *context_lens,
                            int32_t page_size, float scale, int32_t window, int32_t sinks,
                            void *out, pa_shape shape, void *stream);

/*
 * The dispatch of the two: pa_decode_window or pa_prefill_window, by
 * pa_attention_route's rule on the keys a row can reach (the smaller of
 * max_context_len, where known, and sinks + window + L). workspace:
 * pa_attention_window_workspace_bytes bytes (0: none needed, or invalid sizes), any
 * contents; calls that share one must not overlap on the GPU. The decode route
 * needs it, 16-byte aligned. On the prefill route it is for head_dim 128, pages of
 * at least 8 tokens and groups of at least 2 where whole query tiles would leave
 * SMs idle for long: with it (256-byte aligned) the tiles of keys are spread
 * evenly, as pa_prefill_split does; without it the call is pa_prefill_window.
 */
size_t pa_attention_window_workspace_bytes(pa_shape shape, int32_t page_size,
                                           int32_t max_context_len, int32_t window, int32_t sinks);
pa_status pa_attention_window(const void *query, const void *key_pages, const void *value_pages,
                              const int32_t *block_table, const int32_t *context_lens,
                              int32_t page_size, float scale, int32_t window, int32_t sinks,
                              void *out, pa_shape shape, int32_t max_context_len, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * The dispatch for e4m3 pools (head_dim 128): pa_decode_window_fp8 for L <= 8;
 * otherwise the tokens that some row of the call sees are copied into bf16
 * pages of 128 tokens in the workspace, exactly, and pa_prefill_window's kernel
 * attends over the copies (k_scale in the softmax scale, v_scale in the output),
 * as pa_prefill_fp8 does for full attention. max_context_len bounds
 * context_lens; on the second route a longer entry records
 * PA_DEVERR_CONTEXT_LEN and is cut to the next multiple of 128. On the first
 * route the query is taken in f16, as pa_decode_fp8.
 *   workspace  pa_attention_window_fp8_workspace_bytes bytes (0: invalid
 *              sizes), 256-byte aligned, any contents.
 */
size_t pa_attention_window_fp8_workspace_bytes(pa_shape shape, int32_t page_size,
                                               int32_t max_context_len, int32_t window,
                                               int32_t sinks);
pa_status pa_attention_window_fp8(const void *query, const void *key_pages,
                                  const void *value_pages, const int32_t *block_table,
                                  const int32_t *context_lens, int32_t page_size, float scale,
                                  float k_scale, float v_scale, int32_t window, int32_t sinks,
                                  void *out, pa_shape shape, int32_t max_context_len,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * pa_decode that also accumulates the attention weight of every cached slot,
 * for pa_kv_evict. With w[j] = sum of the softmax weights that the G * L rows
 * of a KV group give to position j (a row that sees no key gives none):
 *   weight_pages[slot of j] = decay * weight_pages[slot of j] + w[j]
 * and = w[j] for the L newest positions (their slots are new) and for every
 * position when decay is 0 (the slots are then not read, so a first call with
 * decay 0, for example over a prompt's last rows, sets a pool up).
 *   weight_pages     [P, H_kv, page_size] fp32, updated in place.
 *   decay            finite, >= 0 (1: plain sum).
 *   max_context_len  > 0, bounds context_lens and sizes the workspace; a longer
 *                    entry records PA_DEVERR_CONTEXT_LEN and is cut to it.
 *   workspace        pa_decode_weights_workspace_bytes(shape, max_context_len)
 *                    bytes (the decode's, 4 bytes per row and position, 8 per
 *                    row), 16-byte aligned, any contents; calls sharing one
 *                    must not overlap on the GPU.
 * Pages shared by requests of one call must not be used here (two requests
 * would update one slot). Weights are summed in fp32, rows in order. Three
 * kernels on `stream`. The e4m3 form takes the query in f16, as pa_decode_fp8.
 */
size_t pa_decode_weights_workspace_bytes(pa_shape shape, int32_t max_context_len);
pa_status pa_decode_weights(const void *query, const void *key_pages, const void *value_pages,
                            float *weight_pages, const int32_t *block_table,
                            const int32_t *context_lens, int32_t page_size, float scale,
                            int causal, float decay, void *out, pa_shape shape,
                            int32_t max_context_len, void *workspace, size_t workspace_bytes,
                            void *stream);
pa_status pa_decode_weights_fp8(const void *query, const void *key_pages, const void *value_pages,
                                float *weight_pages, const int32_t *block_table,
                                const int32_t *context_lens, int32_t page_size, float scale,
                                float k_scale, float v_scale, int causal, float decay, void *out,
                                pa_shape shape, int32_t max_context_len, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * Eviction by accumulated attention weight: cuts every request to at most
 * `keep` cached tokens. For each request and KV head it keeps the first
 * `sinks` positions, the last `recent` ones, and of the positions between
 * those of the highest weight in weight_pages (ties to the lowest position; a
 * NaN counts as below every number, -0 as +0), `keep` in all, and moves their
 * K, V and weight rows, in the order of their positions, to positions
 * 0 .. keep - 1 of dst_block_table's pages. KV heads keep different positions
 * but the same number, so a request has one context length afterwards. A
 * request of `keep` tokens or fewer keeps all of them.
 *   key_pages, value_pages  [P, H_kv, page_size, D] bf16 (_fp8: e4m3 codes,
 *                    head_dim 128); weight_pages [P, H_kv, page_size] fp32.
 *   dst_block_table  [B, dst_max_pages] int32. The block table itself (the same
 *                    address; dst_max_pages is max_pages then, or B is 1): in
 *                    place; slots behind the kept ones keep their contents.
 *                    Another table: pages that no request of the call
 *                    reads and no other entry names (pages shared by requests
 *                    are evicted into fresh ones); an entry that is the
 *                    request's own page of the same place records
 *                    PA_DEVERR_PAGE_ID, and rows around it are not written. At least
 *                    min(keep, max_pages * page_size) tokens wide; entries
 *                    behind the kept rows are not read.
 *   kept             [B, H_kv, keep] int32 out: the kept positions, ascending,
 *                    -1 behind the last.
 *   new_lens         [B] int32 out: min(context_lens, keep). kept and new_lens
 *                    overlap neither each other, the tables nor context_lens.
 *   sinks + recent <= keep.
 *   shape            batch, num_kv_heads, head_dim, num_pages, max_pages.
 * A page id outside the pool (PA_DEVERR_PAGE_ID) counts as lowest weights when
 * choosing, and its rows are not moved. The rotation of a moved key stays that
 * of its token's own position. Two kernels on `stream`.
 */
pa_status pa_kv_evict(void *key_pages, void *value_pages, float *weight_pages,
                      const int32_t *block_table, const int32_t *context_lens,
                      int32_t page_size, int32_t keep, int32_t sinks, int32_t recent,
                      const int32_t *dst_block_table, int32_t dst_max_pages,
                      int32_t *kept, int32_t *new_lens, pa_shape shape, void *stream);
pa_status pa_kv_evict_fp8(void *key_pages, void *value_pages, float *weight_pages,
                          const int32_t *block_table, const int32_t *context_lens,
                          int32_t page_size, int32_t keep, int32_t sinks, int32_t recent,
                          const int32_t *dst_block_table, int32_t dst_max_pages,
                          int32_t *kept, int32_t *new_lens, pa_shape shape, void *stream);

/*
 * 4-bit page pools, with a step of their own for every 32 elements of a row (Reading
 * vLLM's PagedAttention Kernel, 3.2: the write path takes the cache dtype; here the
 * scales follow the data, so none are passed). head_dim 128 only. A pool is
 * [P, H_kv, page_size, 80] bytes; a row's first 64 bytes are its codes (element d in
 * byte d / 2, even d in the low half), then for each group of 32 elements its step s and
 * its least value m as f16: s0 m0 s1 m1 s2 m2 s3 m3. A code c stands for m + s c. Rows that
 * another writer puts into a pool have to keep to what pa_append_kv_q4 can write, s in 0 ..
 * 60 and m in -448 .. 448 (or both NaN): the attention calls form 1024 s and 32 m in f16, and
 * give NaN where those do not fit. pa_gather_kv_q4 reads back any s and m.
 */

/*
 * pa_append_kv for 4-bit pools. Of each group of 32 elements of a new row:
 *   y = f16(min(max(x, -448), 448)),  m = min y,  s = f16(fp32(max y - m) / 15),
 *   code = the integer nearest to (y - m) / s, ties to even, at most 15 (0 where s
 *   is 0). A NaN makes its group's m and s NaN.
 * Same slots, checks and error reporting as pa_append_kv. (Of two tokens with the same
 * slot a row may get codes of the one and steps of the other.)
 */
pa_status pa_append_kv_q4(const void *key, const void *value, void *key_pages, void *value_pages,
                          const int32_t *slot_mapping, int32_t page_size, pa_shape shape,
                          void *stream);

/*
 * pa_gather_kv from 4-bit pools: every request's rows as the bf16 nearest to m + s c
 * (fp32 first) in key_dense, value_dense [B, H_kv, dense_len, 128]. The same table,
 * checks and errors; one kernel on `stream`.
 */
pa_status pa_gather_kv_q4(const void *key_pages, const void *value_pages,
                          const int32_t *block_table, const int32_t *context_lens,
                          int32_t page_size, pa_shape shape, int32_t dense_len, void *key_dense,
                          void *value_dense, void *stream);

/*
 * pa_decode over 4-bit pools, straight from the codes: s c is rounded to f16, m is added in
 * the products' fp32 sums. The query and the softmax weights are taken in f16 (query
 * elements below 65504 in magnitude; below 2^-14 they keep fewer bits). A group whose m
 * and s are NaN gives NaN in a visible slot; slots past a request's context are never
 * read. Any L; K and V are read once per 16 rows (G * L) of a request and KV head.
 *   workspace  pa_decode_q4_workspace_bytes(shape) bytes (0: invalid or unsupported
 *              shape), 16-byte aligned, any contents; calls that share one must
 *              not overlap on the GPU.
 * Other arguments and errors as for pa_decode. Two kernels on `stream`.
 */
size_t pa_decode_q4_workspace_bytes(pa_shape shape);
pa_status pa_decode_q4(const void *query, const void *key_pages, const void *value_pages,
                       const int32_t *block_table, const int32_t *context_lens, int32_t page_size,
                       float scale, int causal, void *out, pa_shape shape, int32_t max_context_len,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * Prefill over 4-bit pools, as pa_prefill_fp8: the tokens that the requests have cached
 * are copied into pages of 128 tokens in the workspace (m + s c, of K rounded to bf16, of
 * V and of the softmax's weights to f16), and pa_attention's prefill kernels attend over
 * the copies. max_context_len bounds
 * context_lens; a longer entry records PA_DEVERR_CONTEXT_LEN and is cut to the next
 * multiple of 128. workspace: pa_prefill_q4_workspace_bytes bytes (0: invalid sizes),
 * 256-byte aligned, any contents; calls that share one must not overlap on the GPU.
 */
size_t pa_prefill_q4_workspace_bytes(pa_shape shape, int32_t max_context_len);
pa_status pa_prefill_q4(const void *query, const void *key_pages, const void *value_pages,
                        const int32_t *block_table, const int32_t *context_lens, int32_t page_size,
                        float scale, int causal, void *out, pa_shape shape,
                        int32_t max_context_len, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * The dispatch of the two: pa_decode_q4 for L <= 8, pa_prefill_q4 otherwise, with the
 * same arguments. workspace: the one that call takes, at least
 * pa_attention_q4_workspace_bytes bytes (0: invalid sizes), 256-byte aligned.
 */
size_t pa_attention_q4_workspace_bytes(pa_shape shape, int32_t max_context_len);
pa_status pa_attention_q4(const void *query, const void *key_pages, const void *value_pages,
                          const int32_t *block_table, const int32_t *context_lens,
                          int32_t page_size, float scale, int causal, void *out, pa_shape shape,
                          int32_t max_context_len, void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * Decode of a batch whose requests share long prefixes, each prefix attended to once for
 * all of them: what pa_decode gives (causal) where request b's positions before
 * prefix_lens[p] lie in prefix p's pages. The rows of all requests of a prefix go through
 * the tensor cores together, so its K and V are read once per 256 of their rows; the
 * few-row kernel reads each request's own keys, and a merge joins the two. (Tables that
 * name the same pages are legal in pa_decode too, and short prefixes then lie in L2: up to
 * about 16000 positions, prefix length times its requests, over all prefixes, that call
 * takes as long or less; from about 32000 this one does.)
 *   prefix_table   [num_prefixes, prefix_pages] int32, the pages of each prefix.
 *   prefix_lens    [num_prefixes] int32, tokens, 0 .. min(prefix_pages * page_size,
 *                  max_prefix_len) (a longer one records PA_DEVERR_CONTEXT_LEN and
 *                  is cut). They need not end a page: a request's own copy of the
 *                  last page holds its tokens behind the prefix.
 *   prefix_starts  [num_prefixes + 1] int32, ascending, within 0 .. B: prefix p belongs
 *                  to requests prefix_starts[p] .. prefix_starts[p + 1] - 1; requests
 *                  before the first or from the last on have none. Where they do not
 *                  ascend PA_DEVERR_PREFIX is recorded and the outputs are numbers
 *                  without meaning.
 *   block_table    entries of pages that lie wholly before a request's prefix_len are
 *                  not read and may hold anything.
 *   context_lens   positions in all, prefix included; a request may be shorter than its
 *                  prefix (or empty): its rows see what they see. (The prefix's values
 *                  go through the products for all its rows, with weights of 0 for
 *                  those that do not see them: an infinity or NaN among the values
 *                  makes NaN of rows that end before it too. Keys that a row does not
 *                  see may hold anything.)
 *   num_prefixes   1 .. 256;  max_prefix_len > 0 bounds prefix_lens and sizes the
 *                  workspace.
 *   workspace      ..._workspace_bytes(shape, page_size, num_prefixes, max_prefix_len)
 *                  bytes (0: invalid or unsupported sizes), 256-byte aligned, any
 *                  contents; calls that share one must not overlap on the GPU.
 * Other arguments and errors as for pa_decode / pa_decode_fp8 / pa_decode_q4. Codes are
 * turned into f16 (e4m3 exactly; a prefix's 4-bit values m + s c rounded once), as are the
 * query and the softmax weights over them. Built for few rows a request; any L is
 * computed. Three kernels on `stream`; where a bf16 pool's pages hold fewer than 8
 * tokens, one more before them copies the prefixes into pages of 128 in the workspace.
 */
size_t pa_decode_prefix_workspace_bytes(pa_shape shape, int32_t page_size, int32_t num_prefixes,
                                        int32_t max_prefix_len);
pa_status pa_decode_prefix(const void *query, const void *key_pages, const void *value_pages,
                           const int32_t *block_table, const int32_t *context_lens,
                           int32_t page_size, float scale, const int32_t *prefix_table,
                           const int32_t *prefix_lens, const int32_t *prefix_starts,
                           int32_t num_prefixes, int32_t prefix_pages, int32_t max_prefix_len,
                           void *out, pa_shape shape, int32_t max_context_len, void *workspace,
                           size_t workspace_bytes, void *stream);
size_t pa_decode_prefix_fp8_workspace_bytes(pa_shape shape, int32_t page_size,
                                            int32_t num_prefixes, int32_t max_prefix_len);
pa_status pa_decode_prefix_fp8(const void *query, const void *key_pages, const void *value_pages,
                               const int32_t *block_table, const int32_t *context_lens,
                               int32_t page_size, float scale, float k_scale, float v_scale,
                               const int32_t *prefix_table, const int32_t *prefix_lens,
                               const int32_t *prefix_starts, int32_t num_prefixes,
                               int32_t prefix_pages, int32_t max_prefix_len, void *out,
                               pa_shape shape, int32_t max_context_len, void *workspace,
                               size_t workspace_bytes, void *stream);
size_t pa_decode_prefix_q4_workspace_bytes(pa_shape shape, int32_t page_size,
                                           int32_t num_prefixes, int32_t max_prefix_len);
pa_status pa_decode_prefix_q4(const void *query, const void *key_pages, const void *value_pages,
                              const int32_t *block_table, const int32_t *context_lens,
                              int32_t page_size, float scale, const int32_t *prefix_table,
                              const int32_t *prefix_lens, const int32_t *prefix_starts,
                              int32_t num_prefixes, int32_t prefix_pages, int32_t max_prefix_len,
                              void *out, pa_shape shape, int32_t max_context_len, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * Synchronises `stream`, then reads and clears the device error word of the
 * current device. *flags (may be NULL) receives the PA_DEVERR_* bits seen
 * since the last call. Returns PA_OK when no bit was set,
 * PA_ERR_DEVICE_TIMEOUT when the timeout bit was set, PA_ERR_DEVICE_BOUNDS
 * for any other bit, PA_ERR_CUDA if synchronising failed.
 */
pa_status pa_get_device_error(void *stream, uint32_t *flags);

/*
 * Host-side page allocator and per-step metadata (host code, no GPU work).
 * One pa_kv_cache is one layer's page pool of num_pages pages of page_size
 * tokens, and the pages each request (seq_id) holds in it (Week 3 Day 4,
 * "Decode Metadata"; Tutorial 13, section 4 "The Request Cache"). Not
 * thread-safe: one host thread per cache at a time.
 *   - pages are handed out freed-first (the last freed page first), else the
 *     lowest page id never handed out;
 *   - pa_kv_cache_plan places new tokens by the tail-fill rule: the next token
 *     goes into the request's tail page while it has room, otherwise into a
 *     new page;
 *   - pa_kv_cache_release returns every page of a request exactly once; a
 *     second release (or an unknown seq_id) is PA_ERR_INVALID_ARG.
 */
typedef struct pa_kv_cache pa_kv_cache;

pa_status pa_kv_cache_create(int32_t num_pages, int32_t page_size, pa_kv_cache **cache);
void pa_kv_cache_destroy(pa_kv_cache *cache);

/* A new request with no tokens; PA_ERR_INVALID_ARG if seq_id exists. */
pa_status pa_kv_cache_add(pa_kv_cache *cache, int64_t seq_id);
pa_status pa_kv_cache_release(pa_kv_cache *cache, int64_t seq_id);

/*
 * Cuts seq_id to its first new_len tokens (0 .. the tokens it has) and gives
 * back the pages behind them, last page first: the host side of pa_kv_evict in
 * place, whose new length min(context length, keep) the host knows without
 * reading the device. The pages may be handed out to work that follows on the
 * same stream. PA_ERR_INVALID_ARG (nothing changed) for an unknown seq_id,
 * another new_len, or one that ends inside a page given back by
 * pa_kv_cache_trim_window. Other pages given back behind the new length stay gone
 * (table entries of -1), and the call does not know the window of the rows to come:
 * a row whose window reaches into such a page reads the entry, which is recorded
 * (PA_DEVERR_PAGE_ID). Where t tokens may be cut again (a draft that is not taken),
 * trim for a window of at least the rows' window + t.
 */
pa_status pa_kv_cache_truncate(pa_kv_cache *cache, int64_t seq_id, int32_t new_len);

/*
 * Gives back the full pages of seq_id that no later row sees through a sliding
 * window of `window` keys and the first `sinks` keys (pa_decode_window's mask, for
 * query rows at positions from the current length on): the host side of the
 * window calls. The pages' block-table entries are -1 from then on; the length
 * and all other positions stay. Call it after the step whose rows still saw
 * them was issued; the pages may be handed out to work that follows on the same
 * stream. A sequence trimmed for one window must not be attended to with a larger
 * one. PA_ERR_INVALID_ARG (nothing changed) for an unknown seq_id, window < 1 or
 * sinks < 0.
 */
pa_status pa_kv_cache_trim_window(pa_kv_cache *cache, int64_t seq_id, int32_t window,
                                  int32_t sinks);

/* Pages not held by any request; -1 on a null cache. */
int32_t pa_kv_cache_free_pages(const pa_kv_cache *cache);
/* Tokens cached for seq_id; -1 if unknown. */
int32_t pa_kv_cache_context_len(const pa_kv_cache *cache, int64_t seq_id);

/*
 * One scheduler step for n requests: request i (seq_ids[i], all distinct and
 * added) gets new_tokens[i] (0 .. l_new) new tokens. Writes, into host
 * arrays:
 *   block_table   [n, max_pages]  the request's page ids in logical order,
 *                                 -1 after the last;
 *   context_lens  [n]             tokens cached after this step;
 *   slot_mapping  [n, l_new]      the flat slot (page * page_size + offset)
 *                                 of each new token in order, -1 after the
 *                                 last (may be NULL when l_new == 0).
 * All or nothing: if the pool runs out of pages or a request would need more
 * than max_pages pages, nothing is changed and PA_ERR_NO_PAGES is returned;
 * bad arguments give PA_ERR_INVALID_ARG, also with nothing changed.
 */
pa_status pa_kv_cache_plan(pa_kv_cache *cache, int32_t n, const int64_t *seq_ids,
                           const int32_t *new_tokens, int32_t max_pages, int32_t l_new,
                           int32_t *block_table, int32_t *context_lens, int32_t *slot_mapping);

/*
 * Snapshot and restore (Tutorial 13, section 7 "Transactional Safety"): a
 * snapshot is a copy of the cache's bookkeeping (free list, fresh-page
 * counter, every request's pages and length). Restoring it puts the cache
 * back as it was when the snapshot was taken, so a step whose K/V write or
 * attention launch failed after pa_kv_cache_plan succeeded can be undone.
 * Pool contents are not part of a snapshot and need no restoring: the rows a
 * failed step wrote lie in free pages or past a request's context length,
 * which no kernel reads. The caller owns the snapshot and frees it with
 * pa_kv_cache_snapshot_destroy; restoring a snapshot of another cache is
 * PA_ERR_INVALID_ARG. A snapshot stays valid after restore (restore it again
 * to roll back again).
 */
typedef struct pa_kv_cache_snapshot pa_kv_cache_snapshot;

pa_status pa_kv_cache_snapshot_take(const pa_kv_cache *cache, pa_kv_cache_snapshot **snapshot);
pa_status pa_kv_cache_restore(pa_kv_cache *cache, const pa_kv_cache_snapshot *snapshot);
void pa_kv_cache_snapshot_destroy(pa_kv_cache_snapshot *snapshot);

/*
 * One scheduler step run from the host in a single call (Week 3 Day 4,
 * "Decode Metadata": the batch's page metadata prepared once per step):
 * pa_kv_cache_plan writes the three tables, packed as block_table [n,
 * max_pages], then context_lens [n], then slot_mapping [n, l_new] (int32),
 * into `host_tables`; one asynchronous copy moves them to `device_tables`;
 * then pa_append_kv writes the new K/V rows and pa_attention (causal, with
 * max_context_len = the largest planned context length) runs over the step,
 * all on `stream`.
 *   host_tables    pinned host memory of at least
 *                  pa_kv_cache_step_table_bytes(n, max_pages, l_new) bytes.
 *                  The copy is asynchronous: the caller must not rewrite this
 *                  region (for example by the next step) before the copy has
 *                  run (use one region per step in flight, or synchronise).
 *   device_tables  device memory of the same size, 4-byte aligned; the
 *                  kernels of this step read it.
 *   key_new, value_new  [n, num_kv_heads, l_new, head_dim] bf16 (device);
 *                  rows past a request's new_tokens[i] are not written.
 *   query, out     [n, num_q_heads, l_new, head_dim] bf16 (device); a request
 *                  with fewer than l_new new tokens has its new tokens in its
 *                  last new_tokens[i] rows (bottom-right causal alignment);
 *                  its earlier rows attend as tokens already cached.
 *   key_pages, value_pages  the layer's pool [num_pages, num_kv_heads,
 *                  page_size, head_dim] bf16, num_pages and page_size as
 *                  given to pa_kv_cache_create.
 *   workspace      as pa_attention (required when the step takes the decode
 *                  route, L <= pa_attention_route's threshold).
 * Returns the plan's status (nothing changed on failure), PA_ERR_CUDA if the
 * copy could not be issued, or the status of pa_append_kv / pa_attention; in
 * the last two cases the plan stays applied and a snapshot taken before the
 * call undoes it.
 */
size_t pa_kv_cache_step_table_bytes(int32_t n, int32_t max_pages, int32_t l_new);
pa_status pa_kv_cache_step(pa_kv_cache *cache, int32_t n, const int64_t *seq_ids,
                           const int32_t *new_tokens, int32_t l_new, int32_t max_pages,
                           void *host_tables, void *device_tables, size_t table_bytes,
                           const void *key_new, const void *value_new, const void *query,
                           void *key_pages, void *value_pages, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, float scale, void *out,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Static, human-readable name of a status code. */
const char *pa_status_string(pa_status status);

/* Library version, e.g. "0.1.0". */
const char *pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
