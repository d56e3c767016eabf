/*
 * combine_route_amd: operators of a whole MoE block.
 *
 * The norms around a block with its gate and residual scale (and their
 * gradients), the experts in 8-bit integers, and the layer of a few tokens.
 * They live in the same library as ep.h's and moe.h's functions
 * (libcombine_route_amd.so) and share their types, error codes,
 * ep_last_error() and moe.h's conventions: every precondition that sizes and
 * pointers allow is checked on the host before anything is enqueued, a call is
 * asynchronous on stream (a hipStream_t; NULL = the default stream), allocates
 * nothing, does not synchronise and can be captured in a HIP graph; buffers
 * are caller-owned, contiguous, on the current device and must not overlap
 * unless an argument says so; results are deterministic bit for bit. No call
 * keeps state: any number of threads and streams may call at once, each with
 * a workspace of its own where one is needed.
 *
 * INT8 rows: value = code * scale, one FP32 scale per row, codes -127 to 127.
 * Rows written here are quantized as follows (amax: the row's largest
 * magnitude, u = max(amax, 2^-100)): scale = u / 127, code = v * (127 / u)
 * rounded to the nearest whole number, ties to even, both in FP32; a row of
 * zeros gets scale 1. A row that holds a NaN gets scale NaN, one that holds
 * an infinity (and no NaN) an infinite scale, both with codes 0, so that
 * every product of the row is NaN. FP8 rows are moe.h's.
 */
#ifndef COMBINE_ROUTE_AMD_MOE_BLOCK_H
#define COMBINE_ROUTE_AMD_MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An element type beside EP_* and MOE_FP32. */
enum { MOE_INT8 = 4 };

/* Norm after a block, its gate and scaled residual, and the norm before the
 * next block:
 *   u   = y * r1 * post_weight   r1 = 1 / sqrt(mean(y^2) + eps)  (y without
 *                                post_weight)
 *   h   = residual_scale * residual + gate * u    (u without a gate)
 *   out = h * r2 * pre_weight    r2 = 1 / sqrt(mean(h^2) + eps)
 * all in FP32; h is rounded for residual_out only, out is of the sum itself.
 *   y             [rows][hidden] of dtype (EP_BF16 or EP_FP16): the block's
 *                 output.
 *   residual      [rows][hidden] of dtype.
 *   residual_out  [rows][hidden]: h, rounded once. May be the residual itself.
 *   post_weight   [hidden] of weight_dtype (dtype itself, or MOE_FP32), or NULL.
 *   gate          [hidden] of weight_dtype, or [rows / gate_rows][hidden], a
 *                 gate for each gate_rows consecutive rows; or NULL.
 *   gate_rows     0 for one gate; else >= 1 and a divisor of rows.
 *   pre_weight    [hidden] of weight_dtype; NULL iff out and codes are.
 *   out           [rows][hidden] of dtype, or NULL. May be y itself.
 *   codes, scales out quantized (of the FP32 value), or both NULL: codes_dtype
 *                 EP_FP8_E4M3: [rows][hidden] E4M3 and [rows][hidden / 128]
 *                 float (hidden % 128 == 0); MOE_INT8: [rows][hidden] int8
 *                 and [rows] float. Looked at with codes alone.
 *   row_counts, group_rows  as moe_rms_norm: only the first row_counts[g] rows
 *                 of group g are read and written.
 * hidden: a multiple of 8, 8 to 32768. residual_scale finite, eps >= 0 and
 * finite. Rows, weights and codes 16-byte aligned, scales and row_counts
 * 4-byte.
 * Errors: EP_ERR_NULL, EP_ERR_ALIGN, EP_ERR_ARG, EP_ERR_SIZE (hidden above
 * 32768, rows whose waves exceed 2^26), EP_ERR_HIP. rows == 0 returns EP_OK
 * whatever the pointers are. */
typedef struct moe_block_norm_args {
    const void *y;
    const void *residual;
    void *residual_out;
    const void *post_weight;
    const void *gate;
    const void *pre_weight;
    void *out;
    void *codes;
    float *scales;
    const int32_t *row_counts;
    int64_t rows;
    int64_t group_rows;
    int64_t gate_rows;
    int32_t hidden;
    int32_t dtype;
    int32_t weight_dtype;
    int32_t codes_dtype;
    float residual_scale;
    float eps;
} moe_block_norm_args_t;

int moe_block_norm(const moe_block_norm_args_t *args, void *stream);

/* Gradients of moe_block_norm, from its y and the h it left in residual_out
 * (its rounding, and a quantization of out, count as the identity). With n1 =
 * y * r1, n2 = h * r2 and mean() over a row:
 *   d2 = grad_out * pre_weight
 *   d  = grad_h + r2 * (d2 - n2 * mean(d2 * n2))
 *   grad_residual    = residual_scale * d
 *   grad_gate        = sum over the gate's rows of d * u
 *   grad_post_weight = sum over rows of d * gate * n1
 *   d1 = d * gate * post_weight
 *   grad_y           = r1 * (d1 - n1 * mean(d1 * n1))  (d * gate without
 *                      post_weight)
 *   grad_pre_weight  = sum over rows of grad_out * n2
 *   grad_h, grad_out  [rows][hidden] of dtype: gradients of residual_out and
 *                 out, either may be NULL (zeros), not both. pre_weight NULL
 *                 iff grad_out is.
 *   h             [rows][hidden]; NULL is allowed without grad_out.
 *   grad_y        [rows][hidden] of dtype. May be y or grad_h itself.
 *   grad_residual [rows][hidden] of dtype, or NULL. May be h or grad_out
 *                 itself.
 *   grad_post_weight, grad_pre_weight  [hidden] float, or NULL; need
 *                 post_weight, pre_weight.
 *   grad_gate     the gate's shape, float, or NULL; needs gate.
 *   workspace     moe_block_norm_backward_workspace_bytes(rows, hidden,
 *                 groups) bytes, groups = rows / gate_rows with a gate of
 *                 several rows, else rows / group_rows with row_counts, else
 *                 1 (with both, gate_rows has to be group_rows). What is
 *                 enough for some number of groups is enough for any other
 *                 of the same rows. May be NULL if no gradient of a weight or
 *                 gate is asked for.
 *                 Overwritten; 16-byte aligned.
 * Rows past a count are neither read nor written and add nothing to the
 * sums; with rows == 0 (EP_OK) nothing is written. hidden and alignment as
 * moe_block_norm. Sums over rows are in FP32 in a fixed order.
 * Errors: as moe_block_norm; EP_ERR_SIZE also for a workspace_bytes that is
 * too small. */
typedef struct moe_block_norm_backward_args {
    const void *y;
    const void *h;
    const void *grad_h;
    const void *grad_out;
    const void *post_weight;
    const void *gate;
    const void *pre_weight;
    void *grad_y;
    void *grad_residual;
    float *grad_post_weight;
    float *grad_gate;
    float *grad_pre_weight;
    void *workspace;
    const int32_t *row_counts;
    int64_t workspace_bytes;
    int64_t rows;
    int64_t group_rows;
    int64_t gate_rows;
    int32_t hidden;
    int32_t dtype;
    int32_t weight_dtype;
    float residual_scale;
    float eps;
} moe_block_norm_backward_args_t;

/* 0 for sizes that the call refuses. */
size_t moe_block_norm_backward_workspace_bytes(int64_t rows, int32_t hidden, int64_t groups);

int moe_block_norm_backward(const moe_block_norm_backward_args_t *args, void *stream);

/* Rows of bf16 / fp16 quantized to INT8 rows with a scale per row (above).
 *   rows          [n_rows][hidden] of dtype (EP_BF16 or EP_FP16).
 *   codes, scales [n_rows][hidden] int8, [n_rows] float.
 *   row_counts, group_rows  as moe_rms_norm: only the first row_counts[g] rows
 *                 of group g are read and written.
 * hidden: a multiple of 8, 8 to 65536; rows and codes 16-byte aligned, scales
 * and row_counts 4-byte. Errors: EP_ERR_NULL, EP_ERR_ALIGN, EP_ERR_ARG,
 * EP_ERR_SIZE, EP_ERR_HIP. n_rows == 0 returns EP_OK whatever the pointers
 * are. */
typedef struct moe_quantize_int8_args {
    const void *rows;
    void *codes;
    float *scales;
    const int32_t *row_counts;
    int64_t n_rows;
    int64_t group_rows;
    int32_t hidden;
    int32_t dtype;
} moe_quantize_int8_args_t;

int moe_quantize_int8(const moe_quantize_int8_args_t *args, void *stream);

/* Grouped product of expert-major INT8 rows with the experts' INT8 weights, a
 * scale per row (token) on one side and per weight row (output channel) on
 * the other: for group g (an expert), row i < min(counts[g], cap) and weight
 * row j,
 *   y[g][i][j] = a_scales[g][i] * (b_scales[g][j] * sum over e of
 *                a[g][i][e] * b[g][j][e])
 * The sum is exact, in 32-bit integers; its conversion to FP32 and the product
 * with b_scales round once each.
 *   MOE_EPILOGUE_ROWS rounds the product with a_scales to FP32 and then to
 * bf16, or at once to fp16. MOE_EPILOGUE_SWIGLU takes weight rows [0, n / 2) as
 * the gate and [n / 2, n) as the up projection, both in FP32, and rounds z =
 * gate / (1 + exp(-gate)) * up (FP32) to out_dtype: the rows that
 * moe_quantize_int8 makes the next product's input of.
 *   a, a_scales   [groups][cap][k] int8, [groups][cap] float: the packed rows
 *                 and scales of a dispatch of INT8 rows (dispatch_dtype
 *                 EP_FP8_E4M3, whose payload it moves as bytes, with one
 *                 4-byte scale a row), or moe_quantize_int8's.
 *   b, b_scales   [groups][n][k] int8, [groups][n] float.
 *   counts        device int32 [groups] (packed_count; a count above cap means
 *                 cap, one below 0 none), or NULL: cap rows each.
 *   out           ROWS: [groups][cap][n] of out_dtype (EP_BF16 or EP_FP16).
 *                 SWIGLU: [groups][cap][n / 2].
 * Codes of -128 are as any other. Rows past a group's count are neither read
 * nor written. k: a positive multiple of 16 up to 65536 (the sum stays below
 * 2^31); n: a positive multiple of 8 (ROWS) or 16 (SWIGLU); n and groups at
 * most 2^20, groups, cap >= 0. A row's result depends on its own inputs
 * alone. a, b and out 16-byte aligned, the rest 4-byte.
 * Errors: EP_ERR_NULL, EP_ERR_ALIGN, EP_ERR_ARG, EP_ERR_SIZE (n, k or groups
 * too large, or groups * cap above 2^31 - 1), EP_ERR_HIP. groups == 0 or cap
 * == 0 returns EP_OK whatever the pointers are. */
typedef struct moe_grouped_gemm_int8_args {
    const void *a;
    const float *a_scales;
    const void *b;
    const float *b_scales;
    const int32_t *counts;
    void *out;
    int32_t groups;
    int32_t cap;
    int32_t n;
    int32_t k;
    int32_t out_dtype;
    int32_t epilogue;
} moe_grouped_gemm_int8_args_t;

int moe_grouped_gemm_int8(const moe_grouped_gemm_int8_args_t *args, void *stream);

/* A whole layer's experts for a few tokens, in two kernels and without a
 * dispatch: for each token t, over the distinct experts e that its slots name
 * (ids outside 0 .. experts - 1 name none), in the order of their first slots,
 *   out[t] = sum of c * down_e (silu(gate_e x_t) * (up_e x_t))
 * c: the FP32 sum in slot order of the weights of the token's slots that name
 * e, 1 without weights; as combine_standard_moe with every expert on hand and
 * no capacity. It reads the weights of the experts that are hit, once each in
 * calls of up to 16 tokens an expert, and nothing else of their size.
 *   x             [tokens][hidden] of dtype (EP_BF16 or EP_FP16), taken as it
 *                 is: neither x nor the hidden rows are quantized.
 *   indices       [tokens][topk] int32.
 *   weights       [tokens][topk] float, or NULL.
 *   gate_up       [experts][2 * inter][hidden] of weight_dtype, gate rows then
 *                 up rows; down [experts][hidden][inter].
 *   gate_up_scales, down_scales  as expert_mlp's or expert_mlp_int8's:
 *                 EP_FP8_E4M3: float per 128 x 128 block, [experts][2 * inter
 *                 / 128][hidden / 128] and [experts][hidden / 128][inter /
 *                 128]; MOE_INT8: float per weight row, [experts][2 * inter]
 *                 and [experts][hidden].
 *   out           [tokens][hidden] of dtype; 0 for a token without experts.
 *   workspace     moe_few_tokens_workspace_bytes(tokens, topk, hidden, inter)
 *                 bytes, 16-byte aligned, overwritten.
 * Products of x and of the hidden rows (as a bf16 value and the bf16 value of
 * its rest, 16 bits) with the weights' codes, both exact in the matrix units'
 * operands, are summed in FP32; scales, silu, c and the sum over experts are
 * FP32 and out is rounded once. A token's result does not depend on the other
 * tokens of the call.
 * tokens 0 to 64, topk 1 to 64, tokens * topk at most 1024; hidden and inter
 * multiples of 128 (EP_FP8_E4M3) or 16 (MOE_INT8) up to 65536; experts 1 to
 * 65536. x, gate_up, down and out 16-byte aligned, the rest 4-byte.
 * Errors: EP_ERR_NULL, EP_ERR_ALIGN, EP_ERR_ARG, EP_ERR_SIZE (a size or
 * workspace_bytes), EP_ERR_HIP. tokens == 0 returns EP_OK whatever the
 * pointers are. */
typedef struct moe_few_tokens_args {
    const void *x;
    const int32_t *indices;
    const float *weights;
    const void *gate_up;
    const float *gate_up_scales;
    const void *down;
    const float *down_scales;
    void *out;
    void *workspace;
    int64_t workspace_bytes;
    int32_t tokens;
    int32_t topk;
    int32_t experts;
    int32_t hidden;
    int32_t inter;
    int32_t dtype;
    int32_t weight_dtype;
} moe_few_tokens_args_t;

/* 0 for sizes that the call refuses. */
size_t moe_few_tokens_workspace_bytes(int32_t tokens, int32_t topk, int32_t hidden, int32_t inter);

int moe_few_tokens(const moe_few_tokens_args_t *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* COMBINE_ROUTE_AMD_MOE_BLOCK_H */
