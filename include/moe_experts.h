/* The routed experts of a MoE decoder layer behind the router (moe_router.h), on B200
 * (sm_100a): the router's choices sorted by expert, token rows brought into that order and
 * back with the routing weights applied (with the gradients of both), rows quantised to
 * 8-bit floating point with a scale for each block of 128, and the block-scaled 8-bit
 * matrix product, plain and grouped by expert. A layer of gated experts is
 *
 *   mla_rmsnorm_router_topk -> mla_moe_sort -> mla_moe_gather (to e4m3)
 *     -> mla_fp8_grouped_matmul (gate | up) -> mla_fp8_quantize (gated)
 *     -> mla_fp8_grouped_matmul (down) -> mla_moe_combine
 *
 * Symbols: T tokens, K choices per token, E experts held by this call's rank (global ids
 * [first_expert, first_expert + E)), R rows of the expert-ordered buffers (their capacity;
 * T * K is always enough), H hidden. A choice outside the held experts (another rank's,
 * or the router's -1) has no row here.
 *
 * 8-bit values are e4m3 (largest finite 448). Scales are fp32. A row's scales lie
 * block-major: scales[b * R + r] belongs to elements [128 b, 128 b + 128) of row r, so the
 * scales a tile of rows needs for one block are contiguous; a weight [N, K] has one scale
 * per 128 x 128 block, [ceil(N / 128), ceil(K / 128)] row-major. The last block of a size
 * that is not a multiple of 128 covers what is left.
 *
 * Element types of the other tensors are MLA_DTYPE_*. Conventions, library and error codes
 * are those of sparse_mla_decode.h: device pointers to contiguous caller-owned memory,
 * asynchronous on `stream`, on the calling host thread's current device, which must be the
 * one that holds the tensors; nothing is enqueued on an error other than MLA_ERR_CUDA.
 * Pointers are 16-byte aligned, those of int32 and fp32 index, offset, weight and scale
 * arrays 4-byte. No call allocates, keeps state between calls or synchronises; every result
 * is the same from run to run (no atomics on floating-point values), and every call can be
 * captured into a CUDA graph.
 *
 * Buffers must not overlap. Row indices and offsets are read on the device: a row index
 * outside [0, R) counts as no row, and offsets are clamped to [0, R] and to their running
 * maximum, so that a wrong table gives wrong values but never an access out of bounds.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { MLA_DTYPE_BF16 = 0, MLA_DTYPE_FP16 = 1, MLA_DTYPE_FP32 = 2 };

#define MLA_MOE_MAX_EXPERTS 1024
#define MLA_MOE_MAX_TOP_K 32

/* Workspace bytes of mla_moe_sort, or 0 if the sizes are outside its limits. Host only. */
size_t mla_moe_sort_workspace_bytes(int n_tokens, int top_k, int n_experts);

/* Sort the choices by expert: a stable counting sort, choices of one expert in the order
 * of topk_idx (token-major).
 *
 *   topk_idx        [n_tokens, top_k] int32 global expert ids
 *   affinities      [n_tokens, n_experts_total] bf16 (the router's), or NULL
 *   n_experts_total width of affinities (not read when affinities is NULL)
 *   first_expert, n_experts   the experts held here
 *   normalize       1: a token's weights are divided by their sum over its top_k choices
 *                   (held here or not), 0: taken as they are
 *   scale           finite factor on every weight
 *   expert_offsets  [n_experts + 1] int32 (written): expert e's rows are
 *                   [expert_offsets[e], expert_offsets[e + 1])
 *   row_of          [n_tokens, top_k] int32 (written): the choice's row, -1 if none
 *   source_of       [n_tokens * top_k] int32 (written): row r holds choice
 *                   source_of[r] = t * top_k + k; -1 behind the last row
 *   weights         [n_tokens, top_k] fp32 (written when affinities is given; else NULL):
 *                   scale * a / (sum of a, or 1), a = affinities[t, topk_idx[t, k]], 0 for
 *                   an id outside [0, n_experts_total); all 0 where the sum is 0
 *   workspace       >= mla_moe_sort_workspace_bytes(...) bytes, 256-byte aligned, for this
 *                   call alone while it runs; may be NULL where that is 0 bytes or
 *                   n_tokens is 0
 *
 * Limits: 1 <= n_experts <= 1024, 1 <= top_k <= 32, n_tokens >= 0 (0: expert_offsets is
 * zeroed), n_tokens * top_k <= 2^30, first_expert >= 0. */
int mla_moe_sort(const int32_t* topk_idx, const void* affinities, int n_tokens, int top_k, int n_experts_total,
                 int first_expert, int n_experts, int normalize, float scale, int32_t* expert_offsets,
                 int32_t* row_of, int32_t* source_of, float* weights, void* workspace, size_t workspace_bytes,
                 void* stream);

/* rows[row_of[t, k]] = x[t] for every choice that has a row; other rows are left as they
 * were. row_of names a row at most once, as mla_moe_sort writes it (what a row named twice
 * holds is not defined). Its gradient is mla_moe_combine with weights NULL.
 *
 *   x       [n_tokens, hidden] of `dtype`
 *   rows    [n_rows, hidden] of `dtype` when scales is NULL; else e4m3, with
 *   scales  [ceil(hidden / 128), n_rows] fp32 (quantised as mla_fp8_quantize does)
 *
 * Limits: hidden a positive multiple of 16, up to 2^30; 1 <= top_k <= 32; n_tokens and
 * n_rows >= 0, n_tokens * top_k <= 2^30, n_tokens * hidden <= 2^42 - 2048 (hidden
 * counted up to the next multiple of 512). */
int mla_moe_gather(const void* x, int dtype, const int32_t* row_of, int n_tokens, int top_k, int hidden, int n_rows,
                   void* rows, float* scales, void* stream);

/* out[t] = sum over the choices of t that have a row, in the order of k, of
 * weights[t, k] * rows[row_of[t, k]] (weights NULL: of the rows), in fp32, rounded once;
 * 0 for a token without rows. A choice without a row is skipped whatever its weight holds.
 *
 *   rows     [n_rows, hidden] of `dtype`
 *   weights  [n_tokens, top_k] fp32, or NULL
 *   out      [n_tokens, hidden] of `dtype` (written)
 *
 * Limits as for mla_moe_gather. */
int mla_moe_combine(const void* rows, int dtype, const int32_t* row_of, const float* weights, int n_tokens,
                    int top_k, int hidden, int n_rows, void* out, void* stream);

/* Gradients of mla_moe_combine:
 *   grad_rows[row_of[t, k]] = weights[t, k] * grad_out[t]   (rows of no choice: left as they were)
 *   grad_weights[t, k]      = <grad_out[t], rows[row_of[t, k]]>, fp32; 0 for a choice without a row
 * row_of names a row at most once, as mla_moe_sort writes it (the gradients of a row named
 * twice are not added up; what grad_rows then holds there is not defined).
 * grad_rows or grad_weights may be NULL when it is not wanted (not both, unless n_rows is 0);
 * weights may be NULL (ones), and rows may be NULL when grad_weights is. */
int mla_moe_combine_backward(const void* grad_out, const void* rows, int dtype, const int32_t* row_of,
                             const float* weights, int n_tokens, int top_k, int hidden, int n_rows, void* grad_rows,
                             float* grad_weights, void* stream);

/* Rows to e4m3 with a scale for each block of 128 values of a row:
 *   amax = max(max |v|, 2^-100), scale = amax / 448, q = e4m3(v * (448 / amax)),
 * in fp32, q rounded to nearest even. A block that holds a NaN or an infinity becomes NaN
 * as a whole. With gated = 0, v is x [n_rows, cols]; with gated = 1, x is
 * [n_rows, 2 * cols] = [g | u] and v = g / (1 + exp(-g)) * u.
 *
 *   valid_rows  device int32, or NULL: only the first *valid_rows rows are read and
 *               written (e.g. &expert_offsets[n_experts])
 *   q           [n_rows, cols] e4m3 (written)
 *   scales      [ceil(cols / 128), n_rows] fp32 (written)
 *
 * Limits: cols a positive multiple of 16, up to 2^29; n_rows >= 0, n_rows * cols <= 2^42 - 2048
 * (cols counted up to the next multiple of 512). */
int mla_fp8_quantize(const void* x, int dtype, int n_rows, int cols, int gated, const int32_t* valid_rows, void* q,
                     float* scales, void* stream);

/* out[m, n] = sum over blocks b of x_scales[b, m] * w_scales[n / 128, b] *
 *             sum over k in block b of x[m, k] * w[n, k],
 * the products of a block exact and summed by the tensor cores in fp32, the blocks added
 * in fp32, rounded once to the output's type.
 *
 *   x         [n_rows, k] e4m3, x_scales [ceil(k / 128), n_rows]
 *   w         [n, k] e4m3, w_scales [ceil(n / 128), ceil(k / 128)]
 *   out       [n_rows, n] of out_dtype (written)
 *   status    device int32 or NULL: MLA_DEV_WAIT_TIMEOUT is OR-ed into it if a bounded
 *             on-device wait gave up (the output is invalid then); never cleared by the call
 *             (read it with mla_get_device_status)
 *
 * A block's factor x_scales * w_scales is rounded to fp32 by itself, so it has to lie in fp32's
 * range.
 *
 * Limits: n and k positive multiples of 16, up to 2^30; n_rows from 0 to 2^30, and
 * (n_rows / 16 + 1) * ceil(n / 128) < 2^30. */
int mla_fp8_matmul(const void* x, const float* x_scales, const void* w, const float* w_scales, int n_rows, int n,
                   int k, void* out, int out_dtype, int32_t* status, void* stream);

/* The same with a weight for each expert: rows [expert_offsets[e], expert_offsets[e + 1])
 * of x are multiplied with w[e]; rows of no expert are left as they were.
 *
 *   w         [n_experts, n, k] e4m3, w_scales [n_experts, ceil(n / 128), ceil(k / 128)]
 *   expert_offsets  [n_experts + 1] int32 on the device
 *
 * Limits: as above, with (n_rows / 16 + n_experts) * ceil(n / 128) < 2^30; 1 <= n_experts <= 1024;
 * n_experts * n < 2^31. */
int mla_fp8_grouped_matmul(const void* x, const float* x_scales, const void* w, const float* w_scales,
                           const int32_t* expert_offsets, int n_rows, int n_experts, int n, int k, void* out,
                           int out_dtype, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
