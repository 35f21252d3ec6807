/*
 * gmm_moe.h -- what stands around the experts' products in one
 * mixture-of-experts layer: the router, tokens sorted by expert and back, and
 * grouped products with bias, activation and residual.  Calls of the same
 * library as gmm.h, under gmm.h's conventions (dense row-major device tensors
 * owned by the caller, workspace, stream, errors), with these additions:
 *  - A token has k choices; choice j of token t is slot t k + j.  T k <= 2^31 - 1024.
 *  - With T = 0 (or M = 0) the tensors of T (or M) rows may be NULL.
 *  - Indices are read on the device.  One outside its range stands for "none"
 *    and never makes a kernel read or write outside the caller's buffers.
 *  - An output overlaps no other tensor of the call, unless a call says that it
 *    may be one of them.
 *
 * A layer, forward:
 *     gmm_route           scores of the experts -> ids and weights [T,k]
 *     gmm_sort_tokens     ids -> group_sizes, row_of [T,k], slot_of [M]
 *     gmm_dispatch        x [T,K] -> the rows in expert order [M,K]
 *     (grouped products of gmm.h, gmm_ffn.h or gmm_bf16_linear)
 *     gmm_combine         results [M,K] -> tokens [T,K]
 * and backward: gmm_combine_bwd, the products' gradients, gmm_combine without
 * weights (the gradient of gmm_dispatch), gmm_route_bwd.
 */
#ifndef GMM_MOE_H_
#define GMM_MOE_H_

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operations of this header, for gmm_workspace_bytes. */
typedef enum {
    GMM_OP_SORT_TOKENS = 32,     /* gmm_sort_tokens: M = T k, the slots; K and N are not read */
    GMM_OP_BF16_LINEAR = 33,     /* gmm_bf16_linear */
    GMM_OP_BF16_LINEAR_BWD = 34  /* gmm_bf16_linear_bwd */
} gmm_moe_op;

/*
 * gmm_get_tile_config of the two products tells which kernel a call runs, in
 * the words of gmm_ffn.h (kernels 1 to 3 for GMM_OP_BF16_LINEAR; for
 * GMM_OP_BF16_LINEAR_BWD dX's, in a call for both gradients: 2 to 4, the weight
 * gradient, unless in that launch, as GMM_OP_TGMM_MX8 of N columns).
 */

/* What an expert's score is made of a logit. */
typedef enum {
    GMM_SCORE_SOFTMAX = 0, /* exp(l_e) / sum over all experts of exp(l) */
    GMM_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-l_e)) */
} gmm_score;

typedef enum {
    GMM_ACT_NONE = 0,
    GMM_ACT_RELU = 1,     /* max(z, 0); a NaN stays one, in the value and in the slope */
    GMM_ACT_SILU = 2,     /* z / (1 + exp(-z)) */
    GMM_ACT_GELU = 3,     /* z (1 + erf(z / sqrt 2)) / 2 */
    GMM_ACT_GELU_TANH = 4 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
} gmm_activation;

#define GMM_MAX_TOPK 64

/*
 * gmm_route -- the k experts of every token and their weights.
 * logits: [T,E], GMM_F32 or GMM_BF16.  1 <= k <= min(E, GMM_MAX_TOPK),
 *   E <= GMM_MAX_GROUPS.
 * bias: [E] fp32 or NULL.
 * An expert whose logit is -infinity or NaN is off for that token: its score
 *   is 0 and it is not chosen; +infinity counts as the largest finite number.
 * Choice: the k experts of the largest keys in falling order, equal keys by
 *   the lower index.  Without a bias the key is the logit; with one it is
 *   score + bias, both in 64 bits, and an expert whose key is -infinity or
 *   NaN is not chosen.
 * ids [T,k] int32; -1 where fewer than k experts can be chosen.
 * weights [T,k] fp32, of the scores without bias:
 *   normalize 0: scale * score;
 *   normalize 1: scale * score / (sum of the token's chosen scores).
 *   0 where ids is -1.
 */
GMM_API int gmm_route(const void *logits, int logits_dtype, const float *bias, int64_t T, int64_t E,
                      int64_t k, int score, int normalize, float scale, int32_t *ids, float *weights,
                      void *stream);

/*
 * gmm_route_bwd -- gradient of the weights with respect to the logits, ids
 *   held fixed.  With s the scores, c the scale and dw the weights' gradient:
 *     softmax:             dl_e = c s_e ([e = ids_j] dw_j - sum_i s_i dw_i), every e
 *     sigmoid:             dl_e = c dw_j s_e (1 - s_e)          for e = ids_j, else 0
 *     normalized, q = s_j / sum of chosen s:  dl_e = c q_j (dw_j - sum_i q_i dw_i),
 *                          times 1 - s_e for the sigmoid         for e = ids_j, else 0
 *   Experts that are off, and choices that are -1, take no part.  An expert
 *   named by several choices of a token gets the sum of their gradients.
 * dweights: [T,k] fp32.  logits, ids: as given to and made by gmm_route.
 * dlogits: [T,E], GMM_F32 or GMM_BF16; of the logits' dtype it may be logits
 *   itself.
 */
GMM_API int gmm_route_bwd(const float *dweights, const void *logits, int logits_dtype,
                          const int32_t *ids, int64_t T, int64_t E, int64_t k, int score,
                          int normalize, float scale, void *dlogits, int dlogits_dtype, void *stream);

/*
 * gmm_sort_tokens -- the order of the slots by expert.
 * ids: [T,k] int32.  Experts first .. first + G - 1 are sorted here (all of
 *   them, or those of an expert-parallel rank); a slot with any other id has
 *   no row.
 * Rows 0, 1, ... take the slots in the order of (expert, slot).  A buffer of
 *   M rows holds the first M of them; slots past that have no row, and the
 *   device status word of ws gets GMM_DEV_SUM_GT_M (0 otherwise).
 * group_sizes [G]: rows of each expert (they sum to at most M).
 * row_of [T,k]: the slot's row, or -1.
 * slot_of [M]: the row's slot, or -1 behind the last one.
 * ws: gmm_workspace_bytes(GMM_OP_SORT_TOKENS, T k, 0, 0, G) bytes: the status
 *   block, and counts unless there are few slots and experts; with more than
 *   256 bytes a call needs a workspace of its own until it has finished.
 * The result does not depend on the order in which anything runs.
 */
GMM_API int gmm_sort_tokens(const int32_t *ids, int64_t T, int64_t k, int64_t first, int64_t G,
                            int64_t M, int32_t *group_sizes, int32_t *row_of, int32_t *slot_of,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * gmm_dispatch -- tokens into the sorted order: out[r] = x[slot_of[r] / k], and
 *   zeros where slot_of[r] is none.
 * x: [T,K], out: [M,K], of one dtype, GMM_BF16 or GMM_F32, K a multiple of 8.
 * row_of and slot_of: made by gmm_sort_tokens (one the other's inverse).
 */
GMM_API int gmm_dispatch(const void *x, int dtype, const int32_t *row_of, const int32_t *slot_of,
                         int64_t T, int64_t k, int64_t M, int64_t K, void *out, void *stream);

/*
 * gmm_combine -- results back to their tokens:
 *     out[t] = residual[t] + sum over j of weights[t,j] * y[row_of[t,j]],
 *   slots without a row left out (their weight may be anything), summed in
 *   fp32 in the order of j, the residual first, rounded once.
 * y: [M,K], y_dtype GMM_BF16 or GMM_F32.  weights: [T,k] fp32 or NULL (all 1:
 *   the gradient of gmm_dispatch).  out: [T,K], out_dtype GMM_BF16 or GMM_F32.
 * residual: [T,K] of out_dtype or NULL; it may be out itself.
 * K a multiple of 8.
 */
GMM_API int gmm_combine(const void *y, int y_dtype, const int32_t *row_of, const float *weights,
                        const void *residual, int64_t T, int64_t k, int64_t M, int64_t K, void *out,
                        int out_dtype, void *stream);

/*
 * gmm_combine_bwd -- gradients of gmm_combine (the residual's is dout):
 *     dy[row_of[t,j]] = weights[t,j] * dout[t],
 *     dweights[t,j]   = sum over columns of dout[t] * y[row_of[t,j]]   (fp32),
 *   0 for a slot without a row; rows of dy that no slot owns are zeros.
 * dout: [T,K], dout_dtype GMM_BF16 or GMM_F32.  y (needed for dweights) and dy:
 *   [M,K], y_dtype GMM_BF16 or GMM_F32.  weights: [T,k] fp32 (needed for dy).
 * dy, dweights [T,k] fp32: NULL where not wanted (both: GMM_ERR_NULL).  dy may
 *   be y itself.
 * row_of and slot_of: made by gmm_sort_tokens.  K a multiple of 8.
 */
GMM_API int gmm_combine_bwd(const void *dout, int dout_dtype, const void *y, int y_dtype,
                            const int32_t *row_of, const int32_t *slot_of, const float *weights,
                            int64_t T, int64_t k, int64_t M, int64_t K, void *dy, float *dweights,
                            void *stream);

/*
 * gmm_bf16_linear -- grouped product with its epilogue in one kernel:
 *     pre = lhs . rhs[g] + bias[g],   out = act(pre) + residual,
 *   the sums, the activation and the residual in fp32, out rounded once.  The
 *   few-row form a serving step needs is chosen inside, from M, N and G.
 * lhs: [M,K] bf16.  rhs: [G,K,N] bf16.  K and N multiples of 64.
 * bias: [G,N], bias_dtype GMM_BF16 or GMM_F32, or NULL.
 * act: a gmm_activation.
 * residual: [M,N] of out_dtype, or NULL; it may be out itself.
 * out: [M,N], GMM_BF16 or GMM_F32.
 * pre: NULL, or [M,N] bf16 that receives pre, which the backward pass needs
 *   unless act is GMM_ACT_NONE.
 * Rows at or past the groups' total: out and pre are zeros there, whatever
 *   lhs and residual hold.
 */
GMM_API int gmm_bf16_linear(const void *lhs, const void *rhs, const int32_t *group_sizes, int64_t M,
                            int64_t K, int64_t N, int64_t G, const void *bias, int bias_dtype,
                            int act, const void *residual, void *out, int out_dtype, void *pre,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * gmm_bf16_linear_bwd -- its backward pass (the residual's gradient is dout):
 *     dpre = dout * act'(pre)   (fp32; act' of ReLU is 0 at 0),
 *     dx = dpre . rhs[g]^T,   dw[g] = lhs_g^T dpre_g,   db[g] = column sums of dpre_g,
 *   the products with dpre rounded to bf16 (unless act is GMM_ACT_NONE, where
 *   it is dout) and fp32 accumulation, db summed in fp32 from the unrounded
 *   values; an empty group's dw and db are 0.
 * dout: [M,N] bf16.  pre: [M,N] bf16 as gmm_bf16_linear kept it (not read, and
 *   may be NULL, with GMM_ACT_NONE).  rhs: [G,K,N] bf16 (needed for dx).
 * lhs: [M,K] bf16 (needed for dw).
 * dx [M,K], dw [G,K,N], db [G,N]: each GMM_BF16 or GMM_F32, NULL where not
 *   wanted (all: GMM_ERR_NULL).
 * ws: gmm_workspace_bytes(GMM_OP_BF16_LINEAR_BWD, ...) bytes, the status block,
 *   dpre and partial sums of db; a call needs one of its own until it has finished.
 */
GMM_API int gmm_bf16_linear_bwd(const void *dout, const void *rhs, const int32_t *group_sizes,
                                const void *lhs, const void *pre, int act, int64_t M, int64_t K,
                                int64_t N, int64_t G, void *dx, int dx_dtype, void *dw, int dw_dtype,
                                void *db, int db_dtype, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_MOE_H_ */
