/*
 * Matrix products grouped by expert, for mixture-of-experts layers: one call
 * multiplies every expert's rows by that expert's matrix, and the two
 * gradients of that product.
 *
 * Rows are sorted by group.  `offsets` is a DEVICE array of groups + 1 int64
 * values, 0 <= offsets[0] <= ... <= offsets[groups] <= rows: group g owns the
 * rows offsets[g] .. offsets[g+1] - 1 and may own none.  It is read when the
 * stream executes the call, so the router's counts never visit the host.
 * Offsets that decrease or leave [0, rows] make the call compute nothing, and
 * gemm_sync_status then reports GEMM_ERR_INVALID.
 *
 * gemm_grouped_run     C[r*ldc + j] = sum_{k < K} A[r*lda + k] * B_g(k, j)
 *                      for every row r of every group g and j < N;
 *                      B_g = B + g * stride_b elements, K x N, in the layouts
 *                      of gemm.h.  Rows of C outside the groups are not
 *                      touched.  K = 0 writes zeros to the groups' rows.
 *                      The gradient of A is the same call on dC with the
 *                      other layout and N and K exchanged.
 * gemm_grouped_wgrad   C_g[i*ldc + j] = sum over rows r of g of
 *                      A[r*lda + i] * B[r*ldb + j], i < M, j < N;
 *                      C_g = C + g * stride_c elements.  A group without rows
 *                      gets zeros.  With A the layer's input and B the
 *                      gradient of its output this is the gradient of a
 *                      row-major weight; exchanged, of a column-major one.
 *
 * A value that is not finite stays in its row of C (gemm_grouped_run) or in
 * its group's C (gemm_grouped_wgrad).
 *
 * dtype GEMM_BF16 (BF16 operands, C float or BF16) or GEMM_TF32 (float
 * operands, whose low 13 mantissa bits the multiplier drops; C float); sums
 * are FP32 and BF16 results are rounded once, to nearest even.  c_dtype is
 * GEMM_F32 or GEMM_BF16.  A, B must be aligned to their element size, C to
 * its own.  Operands whose address, pitch or group stride is not a multiple
 * of 16 bytes are first re-packed into the handle's workspace.  At most
 * GEMM_GROUPED_MAX_GROUPS groups; the rows of a matrix times its pitch stay
 * within 2^44 elements and a group stride within 2^37.  Handles, streams, asynchrony, errors and
 * in-kernel time limits are those of gemm_run; results are bit-identical from
 * call to call.
 */
#ifndef DENSE_GEMM_SM100_GB300_GEMM_GROUPED_H
#define DENSE_GEMM_SM100_GB300_GEMM_GROUPED_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_GROUPED_MAX_GROUPS 4096

/* Or-ed to gemm_grouped_wgrad's c_dtype: all of C becomes NaN where the offsets
 * are refused (without the flag C keeps what it held), and while an expired
 * wait of any call on the handle has not been reported by gemm_sync_status (C
 * may be incomplete). */
#define GEMM_GROUPED_NAN_ON_ERROR 0x100

int gemm_grouped_run(gemm_handle_t h, int layout_b, int64_t groups, int64_t rows, int64_t N, int64_t K,
                     const int64_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb,
                     int64_t stride_b, void *C, int64_t ldc, int dtype, int c_dtype, cudaStream_t stream);

int gemm_grouped_wgrad(gemm_handle_t h, int64_t groups, int64_t rows, int64_t M, int64_t N,
                       const int64_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb,
                       void *C, int64_t ldc, int64_t stride_c, int dtype, int c_dtype, cudaStream_t stream);

/* Argument checks of the two calls without touching the GPU: GEMM_OK,
 * GEMM_ERR_INVALID or GEMM_ERR_ALIGNMENT, exactly as the calls would return. */
int gemm_grouped_validate(int layout_b, int64_t groups, int64_t rows, int64_t N, int64_t K,
                          const int64_t *offsets, const void *A, int64_t lda, const void *B, int64_t ldb,
                          int64_t stride_b, const void *C, int64_t ldc, int dtype, int c_dtype);
int gemm_grouped_wgrad_validate(int64_t groups, int64_t rows, int64_t M, int64_t N, const int64_t *offsets,
                                const void *A, int64_t lda, const void *B, int64_t ldb, const void *C,
                                int64_t ldc, int64_t stride_c, int dtype, int c_dtype);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_SM100_GB300_GEMM_GROUPED_H */
