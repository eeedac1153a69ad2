/*
 * Orthogonalised updates: the orthogonal factor of a matrix by Newton-Schulz
 * steps, for optimisers that replace an update by it.
 *
 * gemm_orthogonalise   For each of `batch` matrices G of rows x cols elements
 *                      (element (r, c) of matrix b at G[b*stride_g + r*ldg + c]):
 *
 *                          X = G / (|G| + eps),   |G| the Frobenius norm
 *                          per step:  A = X X^T,  X = a X + (b A + c A A) X
 *
 *                      (with X^T in the place of X where rows > cols: the
 *                      smaller side's products), and O = X, at
 *                      O[b*stride_o + r*ldo + c].  coefficients: a, b, c of
 *                      every step, 3 * steps values on the host.
 *
 * dtype is that of G and O.  GEMM_BF16: the products take X, A and B = bA + cAA
 * in FP16 (11 bits, one product each) with the diagonals of A and B in FP32 and
 * the rest of X in a second FP16 number beside the product, so that what a step
 * adds to the error stays well below BF16's rounding of the result; GEMM_F32:
 * every operand is two FP16 numbers (22 bits), three products each, sums in FP32
 * cut into parts that are added to nearest.  A matrix of zeros gives zeros; one
 * that holds an infinity or a NaN gives NaN, and its neighbours in the batch are
 * not touched by that.
 *
 * FP16 bounds what may come up on the way: singular values of X up to 7.9, and
 * |b| s^2 + |c| s^4 up to 60 for the largest one s (the usual coefficients stay
 * below 1.3 and 8); past that results may be infinite or NaN.  Elements of A off
 * the diagonal below 2^-36 count as zero, so that a step with a = 0 makes zeros of
 * a matrix that lies as far below eps.  There is no other lower bound: a matrix
 * far below eps grows by a every step, as the formula has it.
 *
 * steps is 1 .. GEMM_ORTHO_MAX_STEPS; the coefficients are finite, eps >= 0.
 * rows and cols are at most 2^20.  O may be G itself (same strides); no other
 * overlap is allowed.  The workspace holds the matrices in FP16, twice over:
 * about 8 * rows * cols + 8 * min(rows, cols)^2 bytes a matrix, of as many
 * matrices at a time as fit 4 GB (at least one).  Handles, streams, workspace,
 * asynchrony, errors and in-kernel time limits are those of gemm_run; results
 * are bit-identical from call to call.
 */
#ifndef DENSE_GEMM_SM100_GB300_GEMM_ORTHO_H
#define DENSE_GEMM_SM100_GB300_GEMM_ORTHO_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ORTHO_MAX_STEPS 32

int gemm_orthogonalise(gemm_handle_t h, int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg,
                       int64_t stride_g, void *O, int64_t ldo, int64_t stride_o, int dtype, int steps,
                       const float *coefficients, float eps, cudaStream_t stream);

/* Argument checks without touching the GPU, exactly as the call makes them. */
int gemm_orthogonalise_validate(int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg,
                                int64_t stride_g, const void *O, int64_t ldo, int64_t stride_o, int dtype, int steps,
                                const float *coefficients, float eps);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_SM100_GB300_GEMM_ORTHO_H */
