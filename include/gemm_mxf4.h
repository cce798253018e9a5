/*
 * MXFP4 matrices and their product for NVIDIA GB300 (sm_103a), in the library
 * of gemm_f16.h, with its status codes, options and device status word.
 *
 * An MXFP4 matrix is `batch` matrices of `rows` rows, each row holding k values
 * along the axis that a product contracts.  32 consecutive values of a row
 * share one scale 2^s; a value is held in 4 bits (sign, 2 exponent bits, 1
 * mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times that scale.
 *
 *   s = floor(log2(max |x|)) - 2, within -127 .. 127 (all zero: -127)
 *   value = x * 2^-s rounded to the nearest of the eight, ties to the even
 *           code, magnitudes above 6 to 6, sign kept
 *
 * A block with a NaN or an infinity gets the NaN scale: all of it reads as NaN.
 *
 * Layout, per matrix of the batch:
 *   codes   rows x (16 * ceil(k / 32)) bytes, row-major; value i of a row in
 *           byte i / 2, the even one in the low nibble; values past k are 0.
 *   scales  512-byte tiles of 128 rows x 4 blocks (128 values), tile
 *           (r / 128, b / 4) at ((r / 128) * ceil(blocks / 4) + b / 4) * 512;
 *           in it row r, block b at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4,
 *           as s + 127 (255: NaN).  Padding rows and blocks hold 0.
 * The next matrix of the batch starts where the previous one ends.  Both
 * arrays start at multiples of 16 bytes.
 */
#ifndef GEMM_MXF4_H
#define GEMM_MXF4_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the unquantised side. */
enum { MXF4_F16 = 0, MXF4_BF16 = 1, MXF4_F32 = 2 };

/* Bytes of the two arrays.  GEMM_F16_ERR_INVALID_VALUE unless rows and k are
 * 1 .. GEMM_F16_MAX_DIM, batch at least 1 and the sizes fit 63 bits. */
gemm_f16_status mxf4_sizes(int64_t rows, int64_t k, int64_t batch, int64_t* code_bytes, int64_t* scale_bytes);

/* Quantise x (element type dtype; value (b, r, i) at b * stride_b + r * stride_r
 * + i * stride_k, strides in elements; stride_r and stride_k positive, stride_b
 * not negative).  codes and scales must not overlap x or each other. */
gemm_f16_status mxf4_quantize(const void* x, int dtype, int64_t stride_b, int64_t stride_r, int64_t stride_k,
                              void* codes, void* scales, int64_t rows, int64_t k, int64_t batch, cudaStream_t stream);

/* The values, rounded once to dtype, as a contiguous y[batch][rows][k]. */
gemm_f16_status mxf4_dequantize(const void* codes, const void* scales, void* y, int dtype, int64_t rows, int64_t k,
                                int64_t batch, cudaStream_t stream);

/* C[m, n] = fp16(act(sum_k A[m, k] * B[n, k] + bias[n])): A of M rows, B of N
 * rows, both with K values; fp32 accumulation, one rounding; bias (fp16, N
 * values, or NULL) and act (GEMM_F16_ACT_*) applied in fp32.  ldc >= N in
 * elements.  C must not overlap an input. */
gemm_f16_status gemm_mxf4(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                          const void* bias, int act, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                          cudaStream_t stream);

/* The same product with A in fp16 (element (m, k) at m * stride_am +
 * k * stride_ak), quantised within the call into `work`: mxf4_sizes(M, K, 1)
 * bytes, the scales first and then the codes, 16-byte aligned, the call's own
 * until its kernels have run. */
gemm_f16_status gemm_mxf4_a16(const void* A, int64_t stride_am, int64_t stride_ak, void* work, const void* B_codes,
                              const void* B_scales, const void* bias, int act, void* C, int64_t ldc, int64_t M,
                              int64_t N, int64_t K, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MXF4_H */
