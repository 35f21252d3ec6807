/*
 * gmm_ffn.h -- the gated expert block (forward, serving and training, and
 * backward) and activation checkpoints in 8 bits: calls of the same library
 * as gmm.h, under gmm.h's conventions (dense row-major device tensors owned
 * by the caller, group_sizes read on the device, workspace, stream, errors;
 * rows at or past the groups' total may hold anything on input and are
 * written as zeros on output).  Widths are multiples of 64 here, and with
 * M = 0 the tensors of M rows may be NULL.
 *
 * 8-bit checkpoints ("mx8").  Every 32 consecutive values of a row share one
 * scale byte c (E8M0: 2^(c - 127)), and each value v is kept as the E4M3 code
 * nearest to v / 2^(c - 127), ties to even.  c is the smallest byte with
 * max|v| <= 448 * 2^(c - 127), 0 for an all-zero block; nothing saturates.
 * A NaN has no part in the maximum and reads back as NaN; so does an infinity
 * (the format has none), whose block is scaled by 2^120.
 * Codes are [M,K] bytes, scales [M,K/32] bytes: 8.25 bits a value.  A value
 * read back is exact in bf16 (magnitudes of 1.9375 * 2^127 and more round to
 * 2^128 and read back as infinity).
 */
#ifndef GMM_FFN_H_
#define GMM_FFN_H_

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operations of this header, for gmm_workspace_bytes. */
typedef enum {
    GMM_OP_BF16_SWIGLU = 16,     /* gmm_bf16_swiglu */
    GMM_OP_BF16_SWIGLU_BWD = 17, /* gmm_bf16_swiglu_bwd */
    GMM_OP_TGMM_MX8 = 18         /* tgmm_mx8 */
} gmm_ffn_op;

/*
 * gmm_get_tile_config of these operations (they take no override) tells which
 * kernel a call of this shape runs; lhs_dtype is not read, M at least 1.
 *   kernel  1 few rows: tile_m = 16, 32 or 64 rows, tile_n = 32 or 64 columns
 *             of P, K split over the waves (a call that keeps P as a checkpoint
 *             takes 64 columns);
 *           2 tiles of 128 rows and tile_n = 128 or 256 columns;
 *           3 tiles of at most tile_m rows (up to 160) and 256 columns, fed by
 *             load waves;
 *           4 dX and dw in one launch (GMM_OP_BF16_SWIGLU_BWD), 128 x 128 tiles.
 *   GMM_OP_BF16_SWIGLU_BWD: dX's, in a call for both gradients.  Its weight
 *   gradient, unless in that launch, runs as GMM_OP_TGMM_MX8 of 2N columns.
 */

/*
 * gmm_quantize_mx8 -- x [M,K] (GMM_BF16 or GMM_F32) into an 8-bit checkpoint:
 *   codes q [M,K], scales [M,K/32].  K a multiple of 32.
 */
GMM_API int gmm_quantize_mx8(const void *x, int x_dtype, int64_t M, int64_t K, uint8_t *q,
                             uint8_t *scale, void *stream);

/*
 * gmm_dequantize_mx8 -- the values of a checkpoint, out [M,K], GMM_BF16 or
 *   GMM_F32 (the same values: each is exact in bf16).  K a multiple of 32.
 *   A value below the smallest normal bf16 number (2^-126) may lose bits.
 */
GMM_API int gmm_dequantize_mx8(const uint8_t *q, const uint8_t *scale, int64_t M, int64_t K,
                               void *out, int out_dtype, void *stream);

/*
 * gmm_bf16_swiglu -- the gated expert block's forward in one kernel:
 *     P = lhs . rhs[g],   out = silu(P[:, :N]) * P[:, N:],
 *   silu(z) = z / (1 + exp(-z)), both projections accumulated, and the
 *   activation and product computed, in fp32.  The few-row form a serving
 *   step needs is chosen inside, from M, N and G.
 * lhs: [M,K] bf16.  rhs: [G,K,2N] bf16, the gate columns first.
 * out: [M,N], GMM_BF16 or GMM_F32.
 * What the backward pass needs of P, kept from the fp32 values, in one of
 * two forms (both NULL: not kept):
 *   gu:             [M,2N] bf16;
 *   gu_q, gu_scale: [M,2N] codes and [M,2N/32] scales, an 8-bit checkpoint
 *                   (both or neither: GMM_ERR_NULL).
 * Giving gu and gu_q is GMM_ERR_DTYPE.  K and N multiples of 64.
 */
GMM_API int gmm_bf16_swiglu(const void *lhs, const void *rhs, const int32_t *group_sizes, int64_t M,
                            int64_t K, int64_t N, int64_t G, void *out, int out_dtype, void *gu,
                            uint8_t *gu_q, uint8_t *gu_scale, void *ws, size_t ws_bytes,
                            void *stream);

/*
 * gmm_bf16_swiglu_bwd -- its backward pass.  With (g, u) the kept P,
 *   s = 1 / (1 + exp(-g)):
 *     dP = [dh * u * s (1 + g (1 - s)),  dh * g * s]   (fp32, rounded to bf16)
 *     dx = dP . rhs[g]^T,   dw[g] = lhs_g^T dP_g,
 *   both products with fp32 accumulation; an empty group's dw is 0.  The
 *   rounding of dP, the products' bf16 operand, is in fp32 results too (about
 *   0.0017 of their norm).
 * dh:  [M,N] bf16.  rhs: [G,K,2N] bf16 (needed for dx).
 * The layer's input, needed for dw: lhs [M,K] bf16, or its 8-bit checkpoint
 *   lhs_q [M,K], lhs_scale [M,K/32].
 * P: gu [M,2N] bf16, or its checkpoint gu_q [M,2N], gu_scale [M,2N/32].
 *   (Of each pair of forms exactly one is given: both is GMM_ERR_DTYPE,
 *   none, or half a checkpoint, GMM_ERR_NULL.)
 * dx:  [M,K], dx_dtype GMM_BF16 or GMM_F32, or NULL (not wanted).
 * dw:  [G,K,2N], dw_dtype GMM_BF16 or GMM_F32, or NULL (not wanted).
 * h:   NULL, or [M,N] bf16 that receives the forward's output recomputed
 *      from the kept P (the next product's weight gradient needs it).
 * ws:  gmm_workspace_bytes(GMM_OP_BF16_SWIGLU_BWD, ...) = 256 + 4 M N bytes, the
 *      status block and dP.  It is written and read by the call's kernels, so
 *      a call needs a workspace of its own until it has finished: two calls on
 *      different streams that share one overwrite each other's dP.
 */
GMM_API int gmm_bf16_swiglu_bwd(const void *dh, const void *rhs, const int32_t *group_sizes,
                                const void *lhs, const uint8_t *lhs_q, const uint8_t *lhs_scale,
                                const void *gu, const uint8_t *gu_q, const uint8_t *gu_scale,
                                int64_t M, int64_t K, int64_t N, int64_t G, void *dx, int dx_dtype,
                                void *dw, int dw_dtype, void *h, void *ws, size_t ws_bytes,
                                void *stream);

/*
 * tgmm_mx8 -- weight gradient of a grouped matmul whose input was kept as an
 *   8-bit checkpoint:
 *     dw[g] = sum over rows m of group g of x[m,:]^T dy[m,:],
 *   x the checkpoint's values (exact bf16 operands), fp32 accumulation; an
 *   empty group gives exactly 0.
 * x_q: [M,K] codes.  x_scale: [M,K/32].  dy: [M,N] bf16.
 * dw: [G,K,N], GMM_BF16 or GMM_F32.  K and N multiples of 64.
 */
GMM_API int tgmm_mx8(const uint8_t *x_q, const uint8_t *x_scale, const void *dy,
                     const int32_t *group_sizes, int64_t M, int64_t K, int64_t N, int64_t G, void *dw,
                     int out_dtype, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_FFN_H_ */
