/*
 * 8-bit matrices and their products for NVIDIA GB300 (sm_103a), in the library
 * of gemm_f16.h, with its status codes, options and device status word.
 *
 * An 8-bit matrix is `batch` matrices of `rows` rows, each row holding k values
 * along the axis that a product contracts.  128 consecutive values of a row
 * share one scale 2^s; a value is held as an e4m3 number (sign, 4 exponent
 * bits, 3 mantissa bits; largest 448) times that scale.
 *
 *   s = the smallest exponent with max |x| <= 448 * 2^s, within -127 .. 127
 *       (all zero: -127)
 *   value = x * 2^-s rounded to the nearest e4m3 number, ties to even
 *
 * A block with a NaN or an infinity gets the NaN scale: all of it reads as NaN.
 *
 * Layout, per matrix of the batch:
 *   codes   rows x (128 * ceil(k / 128)) bytes, row-major; values past k are 0.
 *           (Whole lines of memory: with rows of 4112 bytes a 3001 x 2000 x 4097
 *           product took 30 us, 23 with rows of 4096.)
 *   scales  512-byte tiles of 128 rows x 4 blocks (512 values), tile
 *           (r / 128, b / 4) at ((r / 128) * ceil(blocks / 4) + b / 4) * 512;
 *           in it row r, block b at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4,
 *           as s + 127 (255: NaN).  Padding rows and blocks hold 0.
 * The next matrix of the batch starts where the previous one ends.  Both
 * arrays start at multiples of 16 bytes.
 */
#ifndef GEMM_FP8_H
#define GEMM_FP8_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the unquantised side. */
enum { FP8_F16 = 0, FP8_BF16 = 1, FP8_F32 = 2 };

/* Most groups of one grouped product. */
#define GEMM_FP8_MAX_GROUPS 512

/* Bytes of the two arrays.  GEMM_F16_ERR_INVALID_VALUE unless rows and k are
 * 1 .. GEMM_F16_MAX_DIM, batch at least 1 and the sizes fit 63 bits. */
gemm_f16_status fp8_sizes(int64_t rows, int64_t k, int64_t batch, int64_t* code_bytes, int64_t* scale_bytes);

/* Quantise x (element type dtype; value (b, r, i) at b * stride_b + r * stride_r
 * + i * stride_k, strides in elements; stride_r and stride_k positive, stride_b
 * not negative).  codes and scales must not overlap x or each other. */
gemm_f16_status fp8_quantize(const void* x, int dtype, int64_t stride_b, int64_t stride_r, int64_t stride_k,
                             void* codes, void* scales, int64_t rows, int64_t k, int64_t batch, cudaStream_t stream);

/* The values, rounded once to dtype, as a contiguous y[batch][rows][k]. */
gemm_f16_status fp8_dequantize(const void* codes, const void* scales, void* y, int dtype, int64_t rows, int64_t k,
                               int64_t batch, cudaStream_t stream);

/* C[m, n] = act(sum_k A[m, k] * B[n, k] + bias[n]), rounded once to dtype
 * (FP8_F16 or FP8_BF16): A of M rows, B of N rows, both with K values; fp32
 * accumulation; bias (of C's type, N values, or NULL) and act (GEMM_F16_ACT_*)
 * applied in fp32.  ldc >= N in elements.  C must not overlap an input. */
gemm_f16_status gemm_fp8(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                         const void* bias, int act, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                         cudaStream_t stream);

/* The same product with A in fp16 or bf16 (a_dtype; element (m, k) at m *
 * stride_am + k * stride_ak), quantised within the call into `work`:
 * fp8_sizes(M, K, 1) bytes, the scales first and then the codes, 16-byte
 * aligned, the call's own until its kernels have run. */
gemm_f16_status gemm_fp8_a16(const void* A, int a_dtype, int64_t stride_am, int64_t stride_ak, void* work,
                             const void* B_codes, const void* B_scales, const void* bias, int act, void* C, int dtype,
                             int64_t ldc, int64_t M, int64_t N, int64_t K, cudaStream_t stream);

/* The grouped product: the rows of A [rows, K] in consecutive groups, those of
 * group g times matrix g of B (a batch of `groups` matrices [N, K]),
 *
 *   C[m, n] = act(sum_k A[m, k] * B_g[n, k])                     B_up_codes NULL
 *   C[m, n] = act(sum_k A[m, k] * B_g[n, k]) * (sum_k A[m, k] * B_up_g[n, k])
 *
 * group_rows: `groups` int32 row counts on the DEVICE, read when the kernel
 * runs; a count below zero is taken as zero, and rows past the matrix as
 * absent.  Rows of C past the last group's end are left as they were.  groups is
 * 1 .. GEMM_FP8_MAX_GROUPS; rows may be 0. */
gemm_f16_status gemm_fp8_grouped(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                                 const void* B_up_codes, const void* B_up_scales, const int32_t* group_rows, int act,
                                 void* C, int dtype, int64_t ldc, int64_t rows, int64_t groups, int64_t N, int64_t K,
                                 cudaStream_t stream);

/* The same with A in fp16 or bf16, quantised as in gemm_fp8_a16(). */
gemm_f16_status gemm_fp8_grouped_a16(const void* A, int a_dtype, int64_t stride_am, int64_t stride_ak, void* work,
                                     const void* B_codes, const void* B_scales, const void* B_up_codes,
                                     const void* B_up_scales, const int32_t* group_rows, int act, void* C, int dtype,
                                     int64_t ldc, int64_t rows, int64_t groups, int64_t N, int64_t K,
                                     cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_FP8_H */
