/*
 * Tokens in the order of their experts and back for NVIDIA GB300 (sm_103a), in
 * the library of gemm_f16.h, with its status codes, options and device status
 * word: what stands around a grouped product whose rows are (token, expert)
 * choices.
 *
 * tokens x top_k choices are numbered t * top_k + j.  The place of a choice is its
 * rank by expert, then by its own number.  A choice of no expert (an id outside
 * 0 .. experts - 1) has no place, written -1; places past the last group's end
 * belong to no choice, and rows there are left as they were.  One expert may be
 * chosen more than once by a token.
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include <stddef.h>

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits of one call. */
#define MOE_ROUTE_MAX_EXPERTS 512
#define MOE_ROUTE_MAX_TOP_K 32

/* Bytes of workspace of moe_sort (0 where it needs none). */
gemm_f16_status moe_sort_workspace_size(int64_t tokens, int64_t top_k, int64_t experts, size_t* bytes);

/* From ids [tokens, top_k]: rows [tokens, top_k], the place of each choice;
 * order [tokens * top_k], the choice at each place (-1 past the last group);
 * group_rows [experts], the choices of each expert, which gemm_fp8_grouped()
 * takes.  All int32 on the device.  The workspace (256-byte aligned) may hold
 * anything; it is the call's own until its kernels have run.  tokens may be 0:
 * group_rows is then written as zeros. */
gemm_f16_status moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int32_t* rows,
                         int32_t* order, int32_t* group_rows, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream);

/* out[rows[t, j]] = x[t]: x of `tokens` rows of d fp16 or bf16 values (dtype 0 or
 * 1), out of tokens * top_k rows; row strides in elements, at least d. */
gemm_f16_status moe_gather(const void* x, int dtype, int64_t stride_x, const int32_t* rows, int64_t tokens,
                           int64_t top_k, int64_t d, void* out, int64_t stride_out, cudaStream_t stream);

/* The same for rows held in 8 bits (gemm_fp8.h): codes and scales of a tokens x
 * k matrix into those of a (tokens * top_k) x k matrix. */
gemm_f16_status moe_gather_fp8(const void* codes, const void* scales, const int32_t* rows, int64_t tokens,
                               int64_t top_k, int64_t k, void* out_codes, void* out_scales, cudaStream_t stream);

/* out[t] = sum_j weights[t, j] * y[rows[t, j]] over the choices that have a place,
 * in the order of j, fp32, rounded once.  weights: fp32 [tokens, top_k], or NULL
 * for ones, which is moe_gather()'s gradient. */
gemm_f16_status moe_combine(const void* y, int dtype, int64_t stride_y, const int32_t* rows, const float* weights,
                            int64_t tokens, int64_t top_k, int64_t d, void* out, int64_t stride_out,
                            cudaStream_t stream);

/* moe_combine()'s gradient: dy[rows[t, j]] = weights[t, j] * dout[t] (of dout's
 * type), dweights[t, j] = sum_i dout[t, i] * y[rows[t, j], i] (fp32; 0 for a choice
 * without a place). */
gemm_f16_status moe_combine_grad(const void* dout, int dtype, int64_t stride_dout, const void* y, int64_t stride_y,
                                 const int32_t* rows, const float* weights, int64_t tokens, int64_t top_k, int64_t d,
                                 void* dy, int64_t stride_dy, float* dweights, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_H */
