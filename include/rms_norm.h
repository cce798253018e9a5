/*
 * Root-mean-square norm of rows for NVIDIA GB300 (sm_103a), in the library of
 * gemm_f16.h, with its status codes, options and device status word.
 *
 *   h[r, i] = x[r, i] + residual[r, i]         rounded to their type
 *   y[r, i] = h[r, i] / sqrt(sum_i h[r, i]^2 / d + eps) * weight[i]
 *
 * x, residual, weight and sum (h) are fp16 or bf16; the rest is computed in fp32
 * and rounded once, to the same type (y) or to 8 bits (codes and scales of a
 * rows x d matrix as gemm_fp8.h lays it out, what its products take).  A bf16 row
 * whose squares are out of fp32's range is summed 2^80 or 2^-80 times as large.
 */
#ifndef RMS_NORM_H
#define RMS_NORM_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most values of a row. */
#define RMS_NORM_MAX_DIM 32768

/* dtype: FP8_F16 (0) or FP8_BF16 (1).  Rows are contiguous, the row strides in
 * elements and at least d.  residual may be NULL, and sum then is; sum may be
 * the memory of x or of residual with the same row stride, and overlaps no
 * other input.  Either y or codes and scales are given, the others NULL; they
 * overlap nothing else.  eps is finite and not negative.  rows may be 0. */
gemm_f16_status rms_norm(const void* x, int dtype, int64_t stride_x, const void* residual, int64_t stride_residual,
                         const void* weight, float eps, void* sum, int64_t stride_sum, void* y, int64_t stride_y,
                         void* codes, void* scales, int64_t rows, int64_t d, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_H */
