/*
 * moe_fp8.h -- FP8 (e4m3) operators of libmoe_b200 (C ABI): quantisation with one fp32
 * scale per block of 128 and the grouped matrix product of such operands.  Types,
 * status codes and conventions are those of moe.h (device pointers of the current
 * device, validation before any launch, asynchronous on `stream`, capturable).
 *
 * The same format as an expert weight type: moe_shape.w_dtype = MOE_FP8 (moe.h).
 *
 * Format.  A row of activations [K] holds e4m3 values q [K] and fp32 scales
 * s [ceil(K/128)], one per 128 consecutive columns (the last block may be shorter); a
 * weight matrix [N, K] holds q [N, K] and s [ceil(N/128), ceil(K/128)], one scale per
 * 128 x 128 block.  The value is q * s.  Quantisation of a block with largest magnitude
 * amax: s = max(amax, 2^-100) / 448 rounded to fp32, q = the e4m3 value nearest to the
 * real quotient x / s (ties to even); no block overflows, an all-zero block gives zeros.
 * A NaN gives a NaN q (and does not enter amax); an infinity makes the block's scale
 * infinite, its own q NaN and the block's finite values zeros: their q * s is NaN too.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of activations to e4m3: x [rows, K] of dtype MOE_F32 or MOE_BF16 with `pitch`
 * elements from row to row (>= K); q [rows, K] and scales [rows, ceil(K/128)] fp32,
 * both contiguous.  Any K >= 1, any alignment of x's elements; 16-byte aligned rows with
 * K a multiple of 8 (bf16) or 4 (fp32) take the vectorised path.  rows == 0 is a no-op.
 * Errors: MOE_ERR_DTYPE / SHAPE / NULL / ALIGN (x not aligned to its elements, scales
 * not to 4 bytes). */
MOE_API int moe_fp8_quantize(int dtype, int64_t rows, int64_t K, const void *x, int64_t pitch, uint8_t *q,
                             float *scales, void *stream);

/* Weight stacks to e4m3: w [E, N, K] contiguous of dtype MOE_F32 or MOE_BF16; q [E, N, K]
 * and scales [E, ceil(N/128), ceil(K/128)] fp32.  Same errors as moe_fp8_quantize. */
MOE_API int moe_fp8_quantize_weights(int dtype, int64_t E, int64_t N, int64_t K, const void *w, uint8_t *q,
                                     float *scales, void *stream);

/* Bytes of workspace moe_fp8_matmul needs (0 for rows == 0 or invalid arguments,
 * moe_last_error() then says why).  Its first word is the call's device status
 * (moe_debug_status). */
MOE_API size_t moe_fp8_matmul_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t K);

/* Grouped matrix product: the first counts[0] rows are multiplied by matrix 0, the next
 * counts[1] rows by matrix 1, and so on (moe_permute's expert_counts and row order; NULL
 * with E == 1: every row):
 *   y[r, n] = sum_b xs[r, b] ws[e, n/128, b] sum_{k in block b} xq[r, k] wq[e, n, k]
 * in fp32, rounded once to bf16.  xq [rows, K] and wq [E, N, K] e4m3, xs [rows,
 * ceil(K/128)] and ws [E, ceil(N/128), ceil(K/128)] fp32, y [rows, N] bf16, all
 * contiguous.  counts [E] int32 on the device: a negative count is zero, rows past the
 * sum of the counts are not written, counts past `rows` are cut off.
 * K a multiple of 16, N a multiple of 8, E <= 1024; xq, wq and y 16-byte aligned, the
 * workspace 256-byte aligned and used by this call alone until it completes.  rows == 0
 * is a no-op.
 * Results are bitwise reproducible.  Errors: MOE_ERR_SHAPE / UNSUPPORTED / NULL / ALIGN /
 * WORKSPACE before any launch, MOE_ERR_CUDA if a launch fails. */
MOE_API int moe_fp8_matmul(int64_t rows, int64_t E, int64_t N, int64_t K, const uint8_t *xq, const float *xs,
                           const uint8_t *wq, const float *ws, const int32_t *counts, void *y, void *workspace,
                           size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
