/*
 * swiglu_tokens.h -- C ABI of a token's way through a mixture-of-experts layer in training, and of
 * dropout (same library, status codes and conventions as swiglu_mlp.h; element types as in
 * swiglu_ops.h):
 *
 *   gate       the router's logits -> the chosen experts and their weights
 *   sort       the (token, choice) pairs by expert: rows of each expert, the row of each pair
 *   dispatch   tokens to their experts' rows (then swiglu_moe_fwd / _bwd run the experts)
 *   combine    the experts' rows back to the tokens, weighted, with dropout and the residual stream
 *   dropout    the same dropout for a block without experts
 *
 * each with its gradient.  Tensors of rows are bf16, fp16 or fp32 of any width, with rows at any
 * stride; a pointer needs only its element's alignment, and rows on 16-byte boundaries run fastest.
 * No entry point needs a workspace, copies to the host or waits for the device, and each is fit for
 * stream capture.  All sums have a fixed order: the same call returns the same bits on every run.
 * An output may share memory with an input only where it says so; in its place with another row
 * stride or type it is refused (SWIGLU_ERR_INVALID_ARG).
 */
#ifndef SWIGLU_TOKENS_H
#define SWIGLU_TOKENS_H

#include "swiglu_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The choice of experts.  p = softmax(l) over a token's E logits l; the top_k largest are chosen, by
 * falling logit, ties going to the lowest index (NaN logits rank lowest).
 *   logits [T, E]       `type`, row i at element i * ld
 *   ids [T, top_k]      int32 outputs: the chosen experts
 *   gates [T, top_k]    fp32 outputs: their p, divided by the sum of the chosen p when renormalize
 *                       is not 0
 * A logit of minus infinity switches its expert off for that token.  A choice for which no expert is
 * left has id -1 and gate 0, so a token with all experts off (of a padded batch, say) goes nowhere.
 * Infinite and NaN logits give what the formulas give: gates of NaN.
 * 0 <= T < 2^31, 1 <= top_k <= E <= 1024.
 */
swiglu_status swiglu_moe_gate_fwd(const void* logits, int64_t ld, int32_t* ids, float* gates, int64_t T, int64_t E,
                                  int64_t top_k, int renormalize, int type, void* stream);

/*
 * Its gradient.  With q = gates, the forward's (without renormalize the experts' p), g = dgates, and c_j = 1
 * where ids_j is an expert, else 0:
 *   s = sum_j c_j q_j g_j
 *   renormalize:  dlogits_e = sum_{j: ids_j = e} q_j (g_j - s)
 *   else:         dlogits_e = p_e (sum_{j: ids_j = e} g_j - s),   p = softmax(l)
 * The logits are read only without renormalize (NULL is allowed with it).  gates or dgates of
 * choices without an expert are not used.  A token with all experts off has a gradient of zeros.
 *   dlogits [T, E]      `type`, every element written; may be logits itself (the same stride)
 */
swiglu_status swiglu_moe_gate_bwd(const void* logits, int64_t ld, const int32_t* ids, const float* gates,
                                  const float* dgates, void* dlogits, int64_t lddl, int64_t T, int64_t E,
                                  int64_t top_k, int renormalize, int type, void* stream);

/*
 * Stable sort of (token, choice) pairs by expert.
 *   ids [pairs]         int32; values outside 0 .. E - 1 (-1: none) belong to no expert
 *   counts [E]          int32 output: pairs of each expert.  Expert e's rows are
 *                       counts[0] + ... + counts[e-1] and the counts[e] - 1 after it
 *   pos [pairs]         int32 output: the pair's row, -1 where it has no expert.  An expert's pairs
 *                       keep their order.
 * 0 <= pairs < 2^31, 1 <= E <= 1024.
 */
swiglu_status swiglu_moe_sort(const int32_t* ids, int32_t* counts, int32_t* pos, int64_t pairs, int64_t E,
                              void* stream);

/*
 * Tokens to their experts' rows:  rows[pos_tj] = x_t  for every pair whose pos is in 0 .. n_rows - 1.
 *   x [T, D], rows [n_rows, D]   `type`, with row strides
 *   pos [T, top_k]               int32, no row twice (of two pairs with one row either may be left)
 * Rows that no pair has keep what they held.
 * 0 <= T, n_rows < 2^31, 1 <= D < 2^28, 1 <= top_k <= 1024, D * top_k < 2^31 (here and below).
 */
swiglu_status swiglu_moe_dispatch_fwd(const void* x, int64_t ldx, const int32_t* pos, void* rows, int64_t ldrows,
                                      int64_t T, int64_t D, int64_t top_k, int64_t n_rows, int type, void* stream);

/*
 * Its gradient:  dx_t = add_t + sum_j drows[pos_tj]  over the pairs whose pos is in 0 .. n_rows - 1,
 * in fp32 by rising j, rounded once.
 *   add [T, D]          `add_type`: `type` or SWIGLU_FP32; NULL: none.  dx may be add itself (the
 *                       same type and stride).
 */
swiglu_status swiglu_moe_dispatch_bwd(const void* drows, int64_t lddrows, const int32_t* pos, const void* add,
                                      int64_t ldadd, void* dx, int64_t lddx, int64_t T, int64_t D, int64_t top_k,
                                      int64_t n_rows, int type, int add_type, void* stream);

/*
 * Dropout: each element of a [M, D] tensor is kept with probability P = K / 65536,
 * K = 65536 (1 - p) rounded to the nearest integer (ties to even), and then divided by P; dropped ones are 0 whatever
 * they hold.  Whether element (i, d) is kept depends on (i, d, seed, offset + *step) only: let
 * w = Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as
 * easy as 1, 2, 3", 2011) of the counter (d / 8, i, low and high word of offset + *step) and the key
 * (low and high word of seed).  With b = d % 8 the element's 16 bits are the low (b even) or high (b
 * odd) half of w[b / 2], and it is kept where they are below K.  The mask is computed where it is used
 * and never stored; the gradient's call with the same seed and offset has the same mask.
 *   p                   0 <= p <= 1.  Up to 2^-17: no dropout; from 1 - 2^-17 on everything is dropped
 *   seed, offset        any 64 bits; one (seed, offset) for each mask
 *   step                device int64, or NULL: added to offset (modulo 2^64), read on the device, so
 *                       that a captured graph can have another mask on every replay
 */

/*
 * The experts' rows back to their tokens:
 *   y_t = residual_t + dropout(sum_j gates_tj rows[pos_tj])   over pairs with pos in 0 .. n_rows - 1
 * summed in fp32 by rising j, rounded once.  Rows and gates of other pairs are not read.
 *   rows [n_rows, D], residual, y [T, D]   `type`; residual NULL: none; y may be residual itself
 *                                          (the same stride)
 *   pos [T, top_k] int32, gates [T, top_k] fp32
 */
swiglu_status swiglu_moe_combine_fwd(const void* rows, int64_t ldrows, const int32_t* pos, const float* gates,
                                     const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t D,
                                     int64_t top_k, int64_t n_rows, int type, double p, uint64_t seed,
                                     uint64_t offset, const int64_t* step, void* stream);

/*
 * Its gradient (the residual's is dy).  With e = dropout(dy):
 *   drows[pos_tj] = gates_tj e_t,   dgates_tj = sum_d e_td rows[pos_tj]_d
 * for the pairs whose pos is in 0 .. n_rows - 1 (no row twice); dgates is 0 for the others, and rows
 * that no pair has keep what they held in drows.
 *   dy [T, D], rows, drows [n_rows, D]   `type`;  dgates [T, top_k] fp32
 */
swiglu_status swiglu_moe_combine_bwd(const void* dy, int64_t lddy, const void* rows, int64_t ldrows,
                                     const int32_t* pos, const float* gates, void* drows, int64_t lddrows,
                                     float* dgates, int64_t T, int64_t D, int64_t top_k, int64_t n_rows, int type,
                                     double p, uint64_t seed, uint64_t offset, const int64_t* step, void* stream);

/*
 * y = residual + dropout(x); its gradient with respect to x is the same call on dy without a residual
 * (or with a gradient to add as residual).
 *   x, residual, y [M, D]   `type`, with row strides; residual NULL: none; y may be x or residual
 *                           itself (the same stride)
 * 0 <= M < 2^31, 1 <= D < 2^28.
 */
swiglu_status swiglu_mlp_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy,
                                 int64_t M, int64_t D, int type, double p, uint64_t seed, uint64_t offset,
                                 const int64_t* step, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIGLU_TOKENS_H */
