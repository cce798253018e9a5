/*
 * A whole mixture-of-experts layer for a few tokens on NVIDIA GB300 (sm_103a),
 * in the library of gemm_f16.h, with its status codes, options and device
 * status word.  Two kernels: one routes the tokens, one runs the experts.
 *
 *   l[t, e]  = sum_i x[t, i] * router[i, e]                        (fp32)
 *   the top_k experts of a token are those of its largest l, equal ones in
 *   index order (a NaN counts as larger than every number)
 *   w[t, j]  = exp(l_j - max l) / sum of the same over the chosen experts
 *              (renormalize) or over all of them
 *   h[t, j]  = act(x[t] gate_e) * (x[t] up_e),   e the token's j-th expert
 *   y[t]     = fp16(sum_j w[t, j] * (h[t, j] down_e))
 *
 * x, router and the experts' fp16 weights are fp16 at any positive strides;
 * products are exact, sums fp32.  With fp16 weights h is held between the
 * projections as an fp16 value plus 2^-11 times another, within 2^-23 of
 * itself or 2^-36 where that is less; a magnitude past the fp16 range becomes
 * an infinity, as in the library's products.  With MXFP4 weights x and h are
 * held as sums of 8 MXFP4 values, within 2^-22.5 of the largest magnitude among
 * the 32 values that share a block with them (i / 32); h keeps fp32's range
 * there, and an infinity or a NaN makes its whole block, and so the token's y,
 * NaN.  An expert that no token chose is not read.
 */
#ifndef MOE_F16_H
#define MOE_F16_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits of one call. */
#define MOE_F16_MAX_TOKENS 64
#define MOE_F16_MAX_EXPERTS 512
#define MOE_F16_MAX_TOP_K 8
#define MOE_F16_MAX_DIM 32768

/* One projection of every expert: E matrices [in, out].
 * MOE_F16_WEIGHT_F16: data is fp16, element (e, i, o) at e * stride_e +
 *   i * stride_i + o * stride_o elements; scales NULL.  Fastest with one of
 *   stride_i, stride_o 1, the same one in all three projections, the other
 *   strides multiples of 8 and data 16-byte aligned; where one projection's are
 *   not, all three are read the slower way (2 to 3 times the time), and value by
 *   value (4 times) where they share no unit stride.
 * MOE_F16_WEIGHT_MXF4: data and scales are the codes and scales of E MXFP4
 *   matrices of `out` rows with `in` values each (gemm_mxf4.h); the strides are
 *   not read. */
enum { MOE_F16_WEIGHT_F16 = 0, MOE_F16_WEIGHT_MXF4 = 1 };
typedef struct {
    int format;
    const void* data;
    const void* scales;
    int64_t stride_e, stride_i, stride_o;
} moe_f16_weight;

/* Bytes of workspace for T tokens of D values, F hidden values, E experts. */
gemm_f16_status moe_f16_workspace_size(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k, size_t* bytes);

/* gate and up: D -> F, down: F -> D, all of one format.  y: T rows of D fp16,
 * ldy elements apart.  weights (fp32) and ids (int32), T x top_k contiguous,
 * receive the routing in order of falling l.  The workspace (256-byte aligned)
 * may hold anything; it is the call's own until the call's kernels have run.
 * Outputs must not overlap inputs, the workspace or each other. */
gemm_f16_status moe_f16(const void* x, int64_t stride_xt, int64_t stride_xi, const void* router, int64_t stride_ri,
                        int64_t stride_re, const moe_f16_weight* gate, const moe_f16_weight* up,
                        const moe_f16_weight* down, int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k,
                        int renormalize, int act, void* y, int64_t ldy, float* weights, int32_t* ids, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_F16_H */
