/*
 * Matrix products in 8-bit integers with one scale for every token (row of A)
 * and every channel (row of B), and the quantisation of floating-point operands.
 *
 * A row of K elements is K signed bytes and one float: element k stands for
 * code(k) * scale.
 *
 *   codes   row r at codes + r*ldq bytes, element k at byte k; ldq >= K.  The
 *           base and the pitch are multiples of 16 bytes (else
 *           GEMM_ERR_ALIGNMENT).  Bytes past K are not written and do not
 *           change results; those up to the next multiple of 16 may be read.
 *   scales  one float a row.
 *
 * gemm_i8_quantise     Quantises `batch` matrices of `rows` x K elements of
 *                      type src_dtype (GEMM_F32 or GEMM_BF16) to batch * rows
 *                      output rows; layouts and strides as for
 *                      gemm_mx4_quantise.  The scale of a row is max |x| / 127
 *                      rounded to FP32; codes are x / scale rounded to nearest,
 *                      ties to even, never outside -127 .. 127.  A row of
 *                      zeros has scale 0; one that holds an infinity or a NaN
 *                      has scale NaN and codes 0.
 * gemm_i8_dequantise   dst[r*ldd + k] = code * scale in FP32, rounded to
 *                      dst_dtype.
 * gemm_i8_run          C[i*ldc + j] = (sum_k a(i, k) * b(j, k)) * sa[i] * sb[j],
 *                      i < M, j < N: both operands hold K values a row (B the
 *                      channels of a column-major weight); all 256 codes may
 *                      occur.  The sum is multiplied by sa[i], the product by
 *                      sb[j], each rounded to FP32 (both have to lie in its
 *                      range).  The sum of the codes' products is exact while
 *                      it fits 24 bits.  Beyond that it is a 32-bit integer,
 *                      rounded once, where M is at most 4 (8) and K at most
 *                      24576 (12288); else an FP32 result is the
 *                      sum of exact parts of 768 products each, rounded to FP32
 *                      as they are added (at most one half step of FP32 each),
 *                      and a BF16 result loses less than 2^-23 of the largest
 *                      partial sum for every 16 products past it.
 * gemm_i8_grouped_run  The same over row groups (see gemm_grouped.h): row r of
 *                      group g is multiplied by rows g*N .. g*N + N - 1 of B.
 *                      Sums are 32-bit integers where rows is at most 1536 and
 *                      twice the groups and K at most 24576.
 *
 * The products run on the tensor cores in FP16, which holds every code exactly,
 * or, where sums are 32-bit integers, on integer dot products.  c_dtype is GEMM_F32
 * or GEMM_BF16.  On the tensor cores A is first converted into the handle's
 * workspace (2 bytes an element), B inside the product.  Handles, streams,
 * asynchrony, errors and in-kernel time limits are those of gemm_run; results are
 * bit-identical from call to call.  The rows of a matrix times a pitch stay
 * within 2^44, and a group's codes below 2^40 bytes.
 */
#ifndef DENSE_GEMM_SM100_GB300_GEMM_I8_H
#define DENSE_GEMM_SM100_GB300_GEMM_I8_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Smallest pitch for rows of K codes, in bytes (a multiple of 16). */
int64_t gemm_i8_code_pitch(int64_t K);

int gemm_i8_quantise(gemm_handle_t h, int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                     int64_t stride, int src_dtype, int8_t *codes, int64_t ldq, float *scales, cudaStream_t stream);

int gemm_i8_dequantise(gemm_handle_t h, int64_t rows, int64_t K, const int8_t *codes, int64_t ldq,
                       const float *scales, void *dst, int64_t ldd, int dst_dtype, cudaStream_t stream);

int gemm_i8_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const int8_t *a_codes, int64_t a_ldq,
                const float *a_scales, const int8_t *b_codes, int64_t b_ldq, const float *b_scales, void *C,
                int64_t ldc, int c_dtype, cudaStream_t stream);

int gemm_i8_grouped_run(gemm_handle_t h, int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                        const int8_t *a_codes, int64_t a_ldq, const float *a_scales, const int8_t *b_codes,
                        int64_t b_ldq, const float *b_scales, void *C, int64_t ldc, int c_dtype, cudaStream_t stream);

/* Argument checks without touching the GPU, as the calls make them (groups = 1
 * and offsets = NULL check gemm_i8_run with rows = M). */
int gemm_i8_quantise_validate(int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                              int64_t stride, int src_dtype, const int8_t *codes, int64_t ldq, const float *scales);
int gemm_i8_dequantise_validate(int64_t rows, int64_t K, const int8_t *codes, int64_t ldq, const float *scales,
                                const void *dst, int64_t ldd, int dst_dtype);
int gemm_i8_validate(int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                     const int8_t *a_codes, int64_t a_ldq, const float *a_scales, const int8_t *b_codes,
                     int64_t b_ldq, const float *b_scales, const void *C, int64_t ldc, int c_dtype);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_SM100_GB300_GEMM_I8_H */
