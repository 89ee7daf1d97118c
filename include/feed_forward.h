/*
 * feed_forward.h -- C ABI of a feed-forward block's operators on GB300
 * (sm_103a), part of libgemm_tn: the gated projection with its backward pass,
 * and 8-bit products with a scale for each block of 128.
 *
 *     H = act(A Bg^T) * (A Bu^T)          gemm_tn_gated
 *     dG, dU from dH, G and U             gated_grad
 *     C = A^T B                           gemm_nt      (a weight's gradient)
 *     Q, S with X ~ Q S                   quantize_e4m3
 *     C = (Qa Sa) (Qb Sb)^T               gemm_tn_e4m3
 *
 * The conventions are gemm_tn.h's: sizes are element counts, pitches (ld*)
 * elements between rows, device pointers are the caller's, work is enqueued on
 * `stream` and the call returns; host-side errors are the return value and
 * nothing is enqueued then; a device watchdog's expiry goes to *d_status.
 * Outputs must not overlap inputs or one another, unless said otherwise; a matrix
 * is the stretch of memory from its first element to its last (so columns of one
 * buffer, side by side, overlap). Every sum is held in fp32, and repeated calls give the same bits. Workspaces
 * (padded copies of operands that the tensor-memory-access engine cannot
 * address: base or pitch not a multiple of 16 bytes) come from
 * gemm_tn_workspace_pool() in stream order.
 */
#ifndef FEED_FORWARD_H_
#define FEED_FORWARD_H_

#include "gemm_tn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x / (1 + exp(-x)), beside gemm_tn_activation's. */
enum { GEMM_TN_ACT_SILU = 3 };

/*
 * gemm_tn_gated -- H = act(A Bg^T) * (A Bu^T), one pass over A.
 * a: [m, k]; b: [2n, k], the gate's n rows Bg, then the other projection's n
 * rows Bu; h: [m, n]; all of dtype, any pitch and 2-byte alignment.
 * activation: GEMM_TN_ACT_RELU, _GELU (erf form) or _SILU. The projections
 * are multiplied as fp32 sums, and H is rounded once.
 * pre: nullable [m, 2n] (pitch ldp), receives A Bg^T and A Bu^T side by side,
 * rounded: what gated_grad needs. k == 0: H and pre are zeros.
 * m, n, k < 2^30.
 */
GEMM_TN_API int gemm_tn_gated(int dtype, int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const void* b,
                              int64_t ldb, void* h, int64_t ldh, void* pre, int64_t ldp, int activation, int* d_status,
                              gemm_tn_stream_t stream);

/*
 * gated_grad -- the gradient of H = act(G) * U, element by element:
 * dG = dH * U * act'(G), dU = dH * act(G), in fp32, rounded once.
 * grad: dH, [m, n]; pre: [m, 2n], G and U side by side (gemm_tn_gated's); out:
 * [m, 2n], dG and dU side by side, so that with gemm_tn_gated's A and B
 *     dA = out B      (gemm_nn with k = 2n)
 *     dB = out^T A    (gemm_nt with m = 2n).
 * out may be pre itself (same pointer and pitch). relu's slope at zero is 0.
 */
GEMM_TN_API int gated_grad(int dtype, int64_t m, int64_t n, const void* grad, int64_t ldg, const void* pre, int64_t ldp,
                           void* out, int64_t ldo, int activation, gemm_tn_stream_t stream);

/*
 * gemm_nt -- C[i][j] = sum_k A[k][i] * B[k][j]: C = A^T B with a: [k, m], b:
 * [k, n] of dtype, the summed dimension outermost, read in that layout.
 * c: [m, n] of out_dtype, GEMM_TN_OUT_INPUT or GEMM_TN_OUT_F32. accumulate
 * (fp32 only): the product is added to C, as a gradient is summed over steps.
 * k == 0: C is zeros (accumulate: left as it is).
 */
GEMM_TN_API int gemm_nt(int dtype, int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const void* b,
                        int64_t ldb, void* c, int64_t ldc, int out_dtype, int accumulate, int* d_status,
                        gemm_tn_stream_t stream);

/* Element type of quantize_e4m3's input, and of gemm_tn_e4m3's output. */
enum gemm_tn_element { GEMM_TN_ELEM_F16 = 0, GEMM_TN_ELEM_BF16 = 1, GEMM_TN_ELEM_F32 = 2 };

/*
 * quantize_e4m3 -- X as e4m3 values and a power of two for each block of them.
 * x: [rows, cols] of src_type (gemm_tn_element), pitch ldx. q: e4m3 bytes, [rows, cols]
 * or, with transpose, [cols, rows] (X^T), pitch ldq. A block is 128 elements
 * along a line of q (the last may be shorter) and block_lines lines, 1 or 128:
 * its scale, the least power of two that brings the block's largest finite
 * magnitude to 448 at most (1 for a block of zeros, never less than 2^-126),
 * goes to scale[line / block_lines * s_line + block * s_blk]. q is the
 * quotient, which is exact, rounded to the nearest e4m3 (ties to even);
 * infinities and NaN become NaN and do not count towards the scale.
 * x is aligned to its element.
 */
GEMM_TN_API int quantize_e4m3(int src_type, int64_t rows, int64_t cols, const void* x, int64_t ldx, void* q,
                              int64_t ldq, float* scale, int64_t s_line, int64_t s_blk, int block_lines, int transpose,
                              gemm_tn_stream_t stream);

/*
 * gemm_tn_e4m3 -- C[i][j] = sum over blocks of 128 of K of
 * sa[i][block] * sb[j][block] * sum over the block of A[i][k] * B[j][k].
 * a: [m, k], b: [n, k] e4m3 with 16-byte-aligned bases and pitches (else
 * GEMM_TN_ERR_MISALIGNED). a_scale[i * as_row + block * as_blk]: fp32.
 * b_scale likewise, for every row of b (b_block_rows 1) or for 128
 * rows together, b_scale[j / 128 * bs_row + block * bs_blk] (b_block_rows 128).
 * Fastest with as_row == 1 (and bs_row == 1 where b_block_rows is 1).
 * Products of a block are summed by the tensor core, the blocks in fp32: that sum
 * times the two scales' product, which is taken first. Scales may have any values;
 * where their product leaves fp32's range it is an infinity or zero, and so treated.
 * c: [m, n] of out_type (gemm_tn_element), aligned to its element; accumulate (fp32 only): added
 * to C. k == 0 as in gemm_nt.
 */
GEMM_TN_API int gemm_tn_e4m3(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const float* a_scale,
                             int64_t as_row, int64_t as_blk, const void* b, int64_t ldb, const float* b_scale,
                             int64_t bs_row, int64_t bs_blk, int b_block_rows, void* c, int64_t ldc, int out_type,
                             int accumulate, int* d_status, gemm_tn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FEED_FORWARD_H_ */
