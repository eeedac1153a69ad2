/*
 * Microscaled 4-bit floating point: quantisation, its inverse, and products of
 * quantised operands on the tensor cores.
 *
 * Format (OCP microscaling MXFP4).  A row of K elements is cut into blocks of
 * GEMM_MX4_BLOCK = 32.  A block holds one scale byte s (E8M0: the scale is
 * 2^(s - 127), 0xFF is NaN) and 32 codes of 4 bits (E2M1: sign, then the
 * magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6); the element is code * scale.
 *
 *   codes   row r at codes + r*ldq bytes, two codes a byte, element 2i in the
 *           low half of byte i; ldq >= Kp/2
 *   scales  row r at scales + r*lds bytes, block b at byte b; lds >= Kp/32
 *
 * with Kp = K rounded up to whole blocks; the codes of elements K .. Kp-1 must
 * be zero (gemm_mx4_quantise writes them so).  Both bases and both pitches are
 * multiples of 16 bytes (else GEMM_ERR_ALIGNMENT).  Bytes past Kp/2 and Kp/32
 * in a row are not written and do not change results; of the scales, those in
 * the last 16-byte piece may be read.
 *
 * gemm_mx4_quantise    Quantises `batch` matrices of `rows` x K elements of
 *                      type src_dtype (GEMM_F32 or GEMM_BF16) to batch * rows
 *                      output rows.  GEMM_B_COL_MAJOR: element (r, k) of
 *                      matrix b at src[b*stride + r*ld + k] (activations, and
 *                      column-major weights); GEMM_B_ROW_MAJOR: at
 *                      src[b*stride + k*ld + r] (a row-major K x N weight,
 *                      rows = N; the quantiser turns it).  The scale of a
 *                      block is 2^e, e = max(floor(log2(max |x|)) - 2, -127);
 *                      codes are x / 2^e rounded to nearest, ties to the even
 *                      code, magnitudes past 6 to 6.  A block that holds an
 *                      infinity or a NaN becomes all NaN (scale 0xFF).
 * gemm_mx4_dequantise  dst[r*ldd + k] = the value element (r, k) stands for,
 *                      as float or BF16 (exact in both).
 * gemm_mx4_run         C[i*ldc + j] = sum_k a(i, k) * b(j, k), i < M, j < N:
 *                      both operands quantised along K.  FP32 sums; C float or
 *                      BF16 (c_dtype GEMM_F32 or GEMM_BF16).  The tensor core
 *                      truncates at every addition of 64 products: sums are
 *                      exact while they fit 24 bits (block scales of a row
 *                      within a factor of 16: up to K = 16384 as measured);
 *                      scales spread over 2^16 cost 1.0e-6 of the result's
 *                      norm at K = 4096 and 4.5e-6 at K = 16384.
 * gemm_mx4_grouped_run The same over row groups (see gemm_grouped.h): row r of
 *                      group g is multiplied by rows g*N .. g*N + N - 1 of B.
 *
 * Handles, streams, asynchrony, errors and in-kernel time limits are those of
 * gemm_run.  No call here uses workspace.  The rows of a matrix times a pitch
 * stay within 2^44, and a group's codes below 2^40 bytes.
 */
#ifndef DENSE_GEMM_SM100_GB300_GEMM_MX4_H
#define DENSE_GEMM_SM100_GB300_GEMM_MX4_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_MX4_BLOCK 32

/* Smallest pitches for rows of K elements, in bytes (multiples of 16). */
int64_t gemm_mx4_code_pitch(int64_t K);
int64_t gemm_mx4_scale_pitch(int64_t K);

int gemm_mx4_quantise(gemm_handle_t h, int layout, int64_t batch, int64_t rows, int64_t K, const void *src,
                      int64_t ld, int64_t stride, int src_dtype, void *codes, int64_t ldq, void *scales,
                      int64_t lds, cudaStream_t stream);

int gemm_mx4_dequantise(gemm_handle_t h, int64_t rows, int64_t K, const void *codes, int64_t ldq,
                        const void *scales, int64_t lds, void *dst, int64_t ldd, int dst_dtype,
                        cudaStream_t stream);

int gemm_mx4_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *a_codes, int64_t a_ldq,
                 const void *a_scales, int64_t a_lds, const void *b_codes, int64_t b_ldq, const void *b_scales,
                 int64_t b_lds, void *C, int64_t ldc, int c_dtype, cudaStream_t stream);

int gemm_mx4_grouped_run(gemm_handle_t h, int64_t groups, int64_t rows, int64_t N, int64_t K,
                         const int64_t *offsets, const void *a_codes, int64_t a_ldq, const void *a_scales,
                         int64_t a_lds, const void *b_codes, int64_t b_ldq, const void *b_scales, int64_t b_lds,
                         void *C, int64_t ldc, int c_dtype, cudaStream_t stream);

/* Argument checks without touching the GPU, as the calls make them (groups = 1
 * and offsets = NULL check gemm_mx4_run with rows = M). */
int gemm_mx4_quantise_validate(int layout, int64_t batch, int64_t rows, int64_t K, const void *src, int64_t ld,
                               int64_t stride, int src_dtype, const void *codes, int64_t ldq,
                               const void *scales, int64_t lds);
int gemm_mx4_dequantise_validate(int64_t rows, int64_t K, const void *codes, int64_t ldq, const void *scales,
                                 int64_t lds, const void *dst, int64_t ldd, int dst_dtype);
int gemm_mx4_validate(int64_t groups, int64_t rows, int64_t N, int64_t K, const int64_t *offsets,
                      const void *a_codes, int64_t a_ldq, const void *a_scales, int64_t a_lds,
                      const void *b_codes, int64_t b_ldq, const void *b_scales, int64_t b_lds, const void *C,
                      int64_t ldc, int c_dtype);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_SM100_GB300_GEMM_MX4_H */
