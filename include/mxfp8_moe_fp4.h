/*
 * mxfp8_moe_fp4.h -- second part of libmxfp8.so's C ABI (included by mxfp8.h,
 * whose conventions, status codes and types hold here): the routing of tokens
 * to experts and its gradient, the gradient of the MoE combine, and MXFP4
 * (quantization, dispatch, SwiGLU, dense and grouped products).
 *
 *   mx_moe_route             router logits -> expert ids and weights (what
 *                            mx_moe_dispatch and mx_moe_combine take)
 *   mx_moe_route_bwd         the weights' gradient -> the logits' gradient
 *   mx_moe_combine_bwd       gradients of the expert rows and of the weights
 *   mx_quantize_rowwise_fp4  BF16 -> E2M1 + E8M0, blocks along rows
 *   mx_quantize_colwise_fp4  the same down columns, written transposed
 *   mx_dequantize_fp4        E2M1 + E8M0 -> BF16 or FP32
 *   mx_moe_dispatch_fp4      mx_moe_dispatch with MXFP4 rows
 *   mx_swiglu_quantize_fp4   mx_swiglu_quantize with MXFP4 output
 *   mx_gemm_fp4              C = deq(A) . deq(B)^T, FP32 accumulation
 *   mx_grouped_gemm_fp4      the same per MoE expert over row groups
 *
 * MXFP4 (OCP Microscaling Formats (MX) v1.0):
 *   element  E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 in code order 0..7, bit 3 the
 *            sign; no infinities, no NaN.  Two codes a byte, element 2i in
 *            the low half of byte i; leading dimensions of E2M1 buffers are
 *            in BYTES.
 *   scale    E8M0, as MXFP8's, always in the rearranged layout of
 *            mx_scale_swizzle (32 rows x 8 k-blocks = 256 bytes a tile).
 *   rule     amax = max |v| over the 32 elements; c = floor(log2(amax)) - 2 +
 *            127 clamped to [0, 254] (2 = largest E2M1 exponent); every
 *            element is v / 2^(c-127) rounded to nearest, ties to the even
 *            code, magnitudes above 6 clamped to 6; a negative value that
 *            rounds to zero stays -0 (code 8).
 *   special  an all-zero block gets c = 0 and keeps its zeros' signs; a block
 *            holding NaN or Inf gets c = 0xFF (NaN) and every element code 7.
 *   Results are deterministic, byte for byte.
 */
#ifndef MXFP8_MOE_FP4_H
#define MXFP8_MOE_FP4_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx_score {
    MX_SCORE_SOFTMAX = 0, /* s = softmax of the row's logits   */
    MX_SCORE_SIGMOID = 1  /* s = 1 / (1 + exp(-logit))         */
} mx_score;

#define MX_ROUTE_MAX_TOPK 32

/*
 * Routing: each token's topk experts and their weights.
 *   logits     [tokens][ld_logits] of logits_dtype (MX_BF16 or MX_F32)
 *   bias       DEVICE float [num_experts] or null: added to the scores for
 *              the SELECTION only (a load-balancing correction); finite
 *   score      mx_score
 *   num_groups, topk_groups, group_top
 *              the experts form num_groups equal runs of consecutive numbers;
 *              a group's score is the sum of its group_top (1 or 2) largest
 *              selection scores, and only the topk_groups best groups are
 *              chosen from.  (1, 1, 1): no groups.
 *   renormalize  nonzero: the chosen scores are divided by their sum
 *   scale      factor of every weight
 *   mask       DEVICE uint8 [tokens] or null: a token with 0 is not routed
 *              (its logits are not read)
 *   topk_ids   DEVICE int32 [tokens][topk] out: experts by decreasing
 *              selection score, ties to the lowest number
 *   weights    DEVICE float [tokens][topk] out: scale * s, or
 *              scale * s / (sum of the chosen s)
 * Selection score: s + bias formed in 64 bits and compared to 42 bits of its
 * mantissa; without a bias and with group_top 1 the logit itself (the same
 * order, exactly).  An expert whose logit is -inf is never chosen and takes no
 * part in its group's score; with group_top 2 a group with one expert left ranks
 * below every group with more, among such groups by that expert's score, and a
 * group with none ranks last; groups of equal score rank by number.  Where
 * fewer than topk can be chosen, the remaining ids are -1 (which mx_moe_dispatch
 * does not route) and their weights 0, as for a masked token.  The dispatched
 * rows of such a batch end below tokens*topk: mx_grouped_gemm_fp4 takes their
 * offsets, mx_grouped_gemm asks for an end at M_total.  Renormalized weights are
 * formed from score ratios, so they sum to scale however small the chosen scores
 * are.
 * NaN and +inf: a NaN logit ranks above every number and, where logits are
 * compared, +inf next.  Where scores are compared (a bias, or group_top 2), a
 * softmax row that holds a NaN or +inf has no scores and ranks by its logits in
 * that order, without the bias; a sigmoid's +inf has the score 1.  The weights
 * they take part in are NaN (except +inf's sigmoid, which is 1), the ids stay in
 * range.
 * Requirements: tokens >= 0, num_experts in 1..1024, 1 <= topk <=
 * min(MX_ROUTE_MAX_TOPK, topk_groups * num_experts / num_groups),
 * num_experts % num_groups == 0, 1 <= topk_groups <= num_groups, group_top 1
 * or 2 and at most num_experts / num_groups, ld_logits >= num_experts, scale
 * finite (else MX_ERR_INVALID_ARG, or MX_ERR_UNSUPPORTED above 1024 experts,
 * topk 32, 64 groups or 2^26 - 4 tokens, or for a leading dimension from 2^28);
 * pointers aligned to their elements (else MX_ERR_ALIGN);
 * outputs overlap nothing (else MX_ERR_OVERLAP).
 */
mx_status mx_moe_route(const void *logits, int logits_dtype, int64_t tokens, int64_t num_experts, int64_t ld_logits,
                       const float *bias, int score, int64_t num_groups, int64_t topk_groups, int64_t group_top,
                       int64_t topk, int renormalize, float scale, const uint8_t *mask, int32_t *topk_ids,
                       float *weights, void *stream);

/*
 * Gradient of mx_moe_route's weights with respect to the logits, the choice
 * held fixed (neither the bias nor the groups take part):
 *   with s the scores, S the sum of the chosen ones, g = d_weights:
 *   ds_j = scale * (g_j - sum_k g_k s_k / S) / S   renormalized, else scale * g_j
 *   sigmoid: dx_j = ds_j s_j (1 - s_j);  softmax: dx_i = s_i (ds_i - sum_j ds_j s_j)
 *   topk_ids   DEVICE int32 [tokens][topk] as mx_moe_route wrote them; ids
 *              outside [0, num_experts) take no part; an id that stands
 *              twice in a row counts twice
 *   d_weights  DEVICE float [tokens][topk]
 *   d_logits   [tokens][ld_d] of logits_dtype out: all num_experts columns of
 *              every row are written (zeros where nothing flows: all of a row
 *              without a valid id, a masked token's, whose logits are not read),
 *              computed in FP32 and rounded once
 * Requirements as mx_moe_route's, with topk in 1..MX_ROUTE_MAX_TOPK and
 * ld_d >= num_experts.
 */
mx_status mx_moe_route_bwd(const void *logits, int logits_dtype, int64_t tokens, int64_t num_experts,
                           int64_t ld_logits, int score, int64_t topk, int renormalize, float scale,
                           const int32_t *topk_ids, const float *d_weights, void *d_logits, int64_t ld_d,
                           void *stream);

/*
 * Gradients of mx_moe_combine, out[t] = sum_j weights[t][j] * y[slot[t][j]]:
 *   dy[slot[t][j]] = weights[t][j] * d_out[t]           (one rounding to BF16)
 *   d_weights[t][j] = sum_h d_out[t][h] * y[slot[t][j]][h]   (FP32; 0 where
 *                     slot is -1)
 *   d_out      BF16 [tokens][ld_dout]
 *   y          BF16 [tokens*topk][ld_y], mx_moe_combine's input
 *   slot, weights  as mx_moe_combine's
 *   dy         BF16 [tokens*topk][ld_dy] out, or null (not wanted): rows that
 *              no slot names keep their bytes (they belong to no expert)
 *   d_weights  DEVICE float [tokens][topk] out, or null (not wanted; y may
 *              then be null too).  The sum's order depends on hidden, tokens
 *              and the device's compute-unit count only.
 * dy is the expert down projection's output gradient: mx_quantize_dual_grouped
 * and the grouped products take it as it is.  Slots are distinct
 * (mx_moe_dispatch's are); where two name one row, that row holds one of the
 * two values.  Slots outside [0, tokens*topk) are skipped.
 * Requirements: tokens, hidden >= 0, topk >= 1, tokens * topk and hidden < 2^30 (else
 * MX_ERR_INVALID_ARG); hidden % 8 == 0 (else MX_ERR_SHAPE); d_out, y and dy
 * 16-byte aligned rows (ld % 8; else MX_ERR_ALIGN); outputs overlap nothing
 * (else MX_ERR_OVERLAP).
 */
mx_status mx_moe_combine_bwd(const void *d_out, int64_t tokens, int64_t hidden, int64_t ld_dout, const void *y,
                             int64_t ld_y, const int32_t *slot, const float *weights, int64_t topk, void *dy,
                             int64_t ld_dy, float *d_weights, void *stream);

/*
 * Row-wise MXFP4 quantization, scales rearranged (the operand of a product
 * with K along the rows).
 *   x      BF16 [rows][ld_x]
 *   q      E2M1 [rows][ld_q] out, cols/2 bytes a row
 *   s_swz  tile (rt, kt) of the rearranged scales at byte (rt * s_tiles + kt)
 *          * 256, as mx_quantize_rowwise_swz: the padding rows of the last
 *          32-row tile are not written, and a larger s_tiles writes into the
 *          buffer of a larger operand.  A stack of expert weights [E][N][K]
 *          with N % 32 == 0 is one call with rows = E * N.
 * Requirements: rows, cols >= 0; cols % 32 == 0 (else MX_ERR_SHAPE) and cols
 * % 256 == 0 (else MX_ERR_UNSUPPORTED); ld_x >= cols, ld_q >= cols/2, s_tiles
 * >= cols/256 (else MX_ERR_INVALID_ARG); x and q 16-byte aligned rows (ld_x %
 * 8, ld_q % 16; else MX_ERR_ALIGN); no overlap (else MX_ERR_OVERLAP).
 */
mx_status mx_quantize_rowwise_fp4(const void *x, int64_t rows, int64_t cols, int64_t ld_x, void *q, int64_t ld_q,
                                  void *s_swz, int64_t s_tiles, void *stream);

/*
 * Column-wise MXFP4 quantization of a stack of count tensors, written
 * transposed (the data gradient's weights: expert e's [N][K] becomes [K][N]).
 *   x       BF16 [count*rows][ld_x]: tensor i's rows are i*rows ..
 *   qt      E2M1 [count*cols][ld_qt] out, rows/2 bytes a row: row i*cols + j
 *           encodes column j of tensor i
 *   st_swz  the scales ([count*cols][rows/32]) rearranged, rows/256 tiles a
 *           tile row; tensor i's part starts at i * mx_scale_swizzled_bytes(
 *           cols, rows/32).  Every byte is written.
 * Requirements: count >= 0; rows % 32 == 0 and cols % 32 == 0 (else
 * MX_ERR_SHAPE); rows % 256 == 0 (else MX_ERR_UNSUPPORTED); ld_x >= cols,
 * ld_qt >= rows/2 (else MX_ERR_INVALID_ARG); x and qt 16-byte aligned rows
 * (ld_x % 8, ld_qt % 16), st_swz 4-byte (else MX_ERR_ALIGN); no overlap.
 */
mx_status mx_quantize_colwise_fp4(const void *x, int64_t count, int64_t rows, int64_t cols, int64_t ld_x, void *qt,
                                  int64_t ld_qt, void *st_swz, void *stream);

/*
 * The values an MXFP4 operand stands for: y[i][j] = E2M1(q[i][j]) * 2^(s-127),
 * exact in BF16 and FP32 (NaN where the scale code is 0xFF; magnitudes beyond
 * the largest finite value become infinite: codes the quantizers never write).
 *   q, ld_q, s_swz, s_tiles  as mx_quantize_rowwise_fp4's
 *   y  [rows][ld_y] of y_dtype (MX_BF16 or MX_F32)
 * Requirements as mx_quantize_rowwise_fp4's, with ld_y * element size a
 * multiple of 16.
 */
mx_status mx_dequantize_fp4(const void *q, int64_t rows, int64_t cols, int64_t ld_q, const void *s_swz,
                            int64_t s_tiles, void *y, int64_t ld_y, int y_dtype, void *stream);

/*
 * mx_moe_dispatch with the dispatched rows quantized to MXFP4: the same
 * order, arguments, requirements and workspace (mx_moe_dispatch_workspace_bytes),
 * with q E2M1 [tokens*topk][ld_q] (ld_q >= hidden/2 bytes).
 */
mx_status mx_moe_dispatch_fp4(const void *x, int64_t tokens, int64_t hidden, int64_t ld_x, const int32_t *topk_ids,
                              int64_t topk, int64_t num_experts, int64_t *offsets, int32_t *src_token, int32_t *slot,
                              void *q, int64_t ld_q, void *s_swz, void *workspace, int64_t workspace_bytes,
                              void *stream);

/*
 * mx_swiglu_quantize with MXFP4 output: h is the same, bit for bit; q E2M1
 * [rows][ld_q] (ld_q >= F/2 bytes) and s_swz are mx_quantize_rowwise_fp4 of h.
 */
mx_status mx_swiglu_quantize_fp4(const void *gu, int64_t rows, int64_t F, int64_t ld_gu, void *h, int64_t ld_h,
                                 void *q, int64_t ld_q, void *s_swz, void *stream);

/*
 * Dense MXFP4 product: C[i][j] = sum_k deq(A)[i][k] * deq(B)[j][k], i < M,
 * j < N, accumulated in FP32, written as BF16 (nearest even) or FP32.
 *   a_q  E2M1 [M][ld_a], a_s_swz: its rearranged [M][K/32] scales
 *   b_q  E2M1 [N][ld_b], b_s_swz likewise
 *   c    [M][ld_c] of c_dtype
 * Requirements as mx_gemm's with K % 256 == 0 (else MX_ERR_UNSUPPORTED; K %
 * 32 else MX_ERR_SHAPE) and ld_a, ld_b >= K/2 bytes.  The library estimates
 * the time of each way and takes the least: up to 64 rows (single tokens of a
 * sampler) a kernel that streams B once through all compute units, else tiles
 * of 128x128, 256x128 or 256x256, whose partial last round may be split along
 * K, with FP32 sums in a workspace of mx_gemm_fp4_workspace_bytes bytes (0: none
 * needed; at most 64 MiB).  The way, and with it the sums' order, depends on M,
 * N, K and the device's compute-unit count only.
 */
int64_t mx_gemm_fp4_workspace_bytes(int64_t M, int64_t N, int64_t K, int c_dtype);
mx_status mx_gemm_fp4(int64_t M, int64_t N, int64_t K, const void *a_q, int64_t ld_a, const void *a_s_swz,
                      const void *b_q, int64_t ld_b, const void *b_s_swz, void *c, int64_t ld_c, int c_dtype,
                      void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Grouped MXFP4 product: mx_grouped_gemm's row groups and offsets with MXFP4
 * operands (b_q E2M1 [num_groups][N][K/2 bytes] contiguous).  group_offsets
 * [num_groups] may lie below M_total, as mx_moe_dispatch_fp4 leaves it where
 * assignments are not routed (M_total = tokens*topk): rows of A and its scales
 * outside every group are not used, rows of C not written.  Other requirements
 * as mx_grouped_gemm's with K % 256 == 0.  Few rows per expert (a sampler's
 * step) stream a routed expert's weights once for every 64 of its rows; more
 * take tiles of 128x128 or 256x256.  The rule goes by M_total, num_groups, N, K
 * and the device's compute-unit count, so
 * the offsets are read on the device alone.
 */
mx_status mx_grouped_gemm_fp4(int64_t num_groups, int64_t M_total, int64_t N, int64_t K, const int64_t *group_offsets,
                              const void *a_q, int64_t ld_a, const void *a_s_swz, const void *b_q,
                              const void *b_s_swz, void *c, int64_t ld_c, int c_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_MOE_FP4_H */
