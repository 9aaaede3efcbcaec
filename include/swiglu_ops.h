/*
 * swiglu_ops.h -- C ABI of the operators that stand around the SwiGLU block in training
 * (same library, status codes and conventions as swiglu_mlp.h): layer norm, forward and
 * backward, and the clipping of many gradients by their global norm.
 *
 * Unlike the block's GEMMs these take bf16, fp16 or fp32 tensors of any width, and rows
 * at any stride: a pointer needs only its element's alignment.  Rows on 16-byte boundaries
 * run fastest, then rows off them that start alike in every tensor of a call (contiguous
 * tensors of one odd width do), then others.
 */
#ifndef SWIGLU_OPS_H
#define SWIGLU_OPS_H

#include "swiglu_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors below. */
typedef enum { SWIGLU_BF16 = 0, SWIGLU_FP16 = 1, SWIGLU_FP32 = 2 } swiglu_dtype;

/*
 * Layer norm over the last dimension, with the residual stream's sum fused in.
 *   s    = x + residual               (x alone when residual is NULL)
 *   mean = sum_j s_j / D,   rstd = 1 / sqrt(sum_j (s_j - mean)^2 / D + eps)
 *   y    = (s - mean) * rstd * gamma + beta
 *   x, residual, s, y [M, D]   `type`; row i of x starts at element i * ldx, and so on
 *                              (each row stride at least D).  residual and s go
 *                              together: both NULL or neither.
 *   gamma, beta [D]            `param_type`: `type` or SWIGLU_FP32; NULL = 1 and 0
 *   mean, rstd [M] fp32        saved for the backward; both may be NULL
 * The statistics and y are taken from the unrounded fp32 sum, the deviations in a pass of
 * their own about the mean; rows are held in registers for it, or, past 64 KB (where tensors
 * lie differently, 8192 columns), read three times.  A row's sums are off by at most 53 x 2^-24
 * of the sum of magnitudes at every width; each output is rounded once.
 * 1 <= D < 2^28, 0 <= M < 2^31, eps >= 0.
 * In place: s and y may each be x or residual itself (the same pointer and row stride; then
 * that input is overwritten; with another row stride the call is refused), but not both the
 * same.  No other outputs may overlap inputs or one another.
 */
swiglu_status swiglu_mlp_layer_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                        const void* gamma, const void* beta, void* y, int64_t ldy, void* s,
                                        int64_t lds, float* mean, float* rstd, int64_t M, int64_t D, float eps,
                                        int type, int param_type, void* stream);

/* Bytes of workspace swiglu_mlp_layer_norm_bwd needs: fp32 partial sums of dgamma and
 * dbeta, one plane per CTA, and for D > 6144 two fp32 sums per row.  0 when M or D is
 * not positive. */
size_t swiglu_mlp_layer_norm_bwd_workspace_size(int64_t M, int64_t D);

/*
 * Backward of the layer norm.  With xh = (s - mean) * rstd and g = dy * gamma:
 *   dx     = rstd * (g - sum_j g_j / D - xh * sum_j (g_j xh_j) / D)  (+ dskip)
 *   dgamma = sum_i dy_i xh_i,   dbeta = sum_i dy_i     (over the M rows)
 *   dy, s, dskip, dx [M, D]   `type`, with row strides; s is the forward's normalised
 *                             input (x, or the stored sum).  dskip (NULL: none) is the
 *                             gradient that reaches s past the norm, added before the
 *                             single rounding of dx.
 *   mean, rstd [M] fp32       from the forward
 *   gamma, dgamma, dbeta [D]  `param_type`; gamma NULL = 1; dgamma and dbeta may each be
 *                             NULL (not computed)
 * dgamma and dbeta are summed in fp32 in an order that depends on M, D, the type, dskip's
 * presence and the alignment only: the same call returns the same bits on every run.  M = 0
 * zeroes them.
 * In place: dx may be dy, s or dskip itself (the same pointer and row stride; with another stride
 * the call is refused).
 */
swiglu_status swiglu_mlp_layer_norm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const void* gamma,
                                        const float* mean, const float* rstd, const void* dskip, int64_t ldskip,
                                        void* dx, int64_t lddx, void* dgamma, void* dbeta, int64_t M, int64_t D,
                                        int type, int param_type, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Bytes of workspace swiglu_mlp_clip_grads needs for n tensors: fp64 partial sums. */
size_t swiglu_mlp_clip_grads_workspace_size(int64_t n);

/*
 * Global norm of n gradients and their clipping, without a host synchronisation:
 *   norm  = sqrt(sum_i sum_j in_i[j]^2),   factor = min(1, max_norm / (norm + eps))
 *   out_i = in_i * factor
 *   in, out, counts, types   host arrays of n entries: device pointers (each aligned to
 *                            its element), element counts (0 allowed), swiglu_dtype.
 *                            out_i has in_i's type and count and may be in_i itself (in
 *                            place), but share no memory with another entry's tensors
 *                            (SWIGLU_ERR_INVALID_ARG: one gradient twice in a list would be
 *                            scaled twice); out NULL computes the norm alone.  The arrays
 *                            are read before the call returns.
 *   norm                     device fp32, may be NULL when out is given
 * Squares are fp32 products summed in fp32 16 at a time, then in fp64; where fp32 squares
 * overflow or fall below its normal range they are summed again of scaled elements, so the
 * norm is as precise for the largest and the smallest elements of a type as for others.
 * The sums' order depends on the counts, types and alignment only: the same call returns the
 * same bits on every run.  A norm that is infinite or NaN gives what the formulas give
 * (factor 0, so finite elements become 0 and infinite ones NaN; or NaN everywhere): read
 * `norm` before using the result.  n = 0: norm 0.
 */
swiglu_status swiglu_mlp_clip_grads(const void* const* in, void* const* out, const int64_t* counts, const int* types,
                                    int64_t n, float max_norm, float eps, float* norm, void* workspace,
                                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIGLU_OPS_H */
