/*
 * fp8fg_experts -- the operators around the grouped products of a mixture-of-experts
 * layer on gfx950: routing (with its gradient) and the row segments that the grouped
 * products take, products of few rows with 4-bit weights, and the combination of the
 * experts' rows (with its gradient).
 *
 * Same library, status codes, element types and conventions as fp8fg.h and
 * fp8fg_layer.h: device pointers unless stated otherwise, nothing allocated or
 * retained, no synchronisation, every argument checked on the host before anything is
 * enqueued, no exception across the boundary, capturable in a HIP graph.  Workspaces
 * are the caller's; a call's workspace may be reused once the stream has passed the
 * call.  Outputs must not alias inputs or each other.  No atomics on results: the same
 * bits on every run.
 */
#ifndef FP8FG_EXPERTS_H
#define FP8FG_EXPERTS_H

#include "fp8fg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scores of the experts of a token. */
enum { FP8FG_SCORE_SOFTMAX = 0, FP8FG_SCORE_SIGMOID = 1 };

/*
 * Routing: scores, the k chosen experts of every token and their weights.
 *     s = softmax(z) or sigmoid(z) over the E experts,  c = s + bias
 *     experts[t, 0..k): the k largest c, descending
 *     weights[t, j] = scale * s[experts[t, j]]  (/ the sum of the k chosen s)
 * With groups > 1 only the experts of groups_kept groups are chosen from: a group is E /
 * groups consecutive experts, its score the sum of its group_terms (1 or 2) largest c.
 *
 * Ties go to the lowest index.  Choices compare as real numbers, not as rounded scores:
 * without a bias by the logits, with one (and for sums of two) in fp32, and in 64 bits
 * where fp32 could not tell.
 * An expert whose logit or bias is -infinity is never chosen, and no group whose score
 * is -infinity (one with fewer than group_terms such experts left) is kept; where fewer
 * than k experts are left, the remaining places hold expert -1 with weight 0.  A logit
 * of -infinity has score 0; if all of a token's are, so are all its scores.  A c (without a
 * bias, a logit) that is not a number ranks below all numbers; scores that are not numbers
 * (of a NaN logit, and under softmax all of its token's but those that are 0, as of a logit of
 * +infinity) show in the weights.  Renormalised weights are shares of the scores as real numbers, also where
 * every chosen score is too small for fp32.
 *
 * logits       [T, E] of `dtype`, row pitch ld >= E elements.
 * bias         fp32 [E], or NULL: for the choice only, not in the weights.
 * mask         uint8 [T], or NULL: tokens with 0 (padding) get experts -1, weights 0.
 * score        FP8FG_SCORE_SOFTMAX or FP8FG_SCORE_SIGMOID.
 * experts      out, int32 [T, k].
 * weights      out, fp32 [T, k].
 * scores       out, fp32 [T, E]: s (of every token), or NULL.
 * Requires 1 <= E <= 1024, E % groups == 0, 1 <= groups_kept <= groups <= 64,
 * group_terms <= E / groups where groups are left out, 1 <= k <= 32, k <= groups_kept *
 * E / groups; T < 2^31;
 * scale finite; logits aligned to its element, all others 4-byte (mask: any).  T == 0 is
 * a no-op.
 */
int fp8fg_route_experts(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias,
                        const uint8_t* mask, int score, int64_t groups, int64_t groups_kept, int group_terms,
                        int64_t k, int renormalise, float scale, int32_t* experts, float* weights, float* scores,
                        fp8fg_stream_t stream);

/*
 * Gradient of the routing weights (and of the scores) with respect to the logits; the
 * choice itself passes none.  With p_j = s_j / the sum of the chosen s:
 *     t_j = scale * p_j * (dw_j - sum_i dw_i p_i)   if renormalise, else scale * s_j * dw_j
 *     t and u = dscores * s, per expert:
 *     dz = (t + u) * (1 - s)  for sigmoid,   dz = t + u - s * sum(t + u)  for softmax.
 *
 * dweights     fp32 [T, k];  experts int32 [T, k] as the forward call wrote them (values
 *              outside [0, E) are skipped; a repeated expert counts as often as it occurs).
 * logits, dtype, ld, score, renormalise, scale   as in the forward call.
 * dscores      fp32 [T, E], the gradient that arrives at the scores (of a balance loss,
 *              say), or NULL.
 * dlogits      out, [T, E] of `dtype`.  An expert whose logit is -infinity gets 0, and has p = 0.
 * Requirements as the forward call's.
 */
int fp8fg_route_experts_backward(const float* dweights, const int32_t* experts, const void* logits, int dtype,
                                 int64_t T, int64_t E, int64_t ld, int score, int64_t k, int renormalise, float scale,
                                 const float* dscores, void* dlogits, fp8fg_stream_t stream);

/*
 * Row segments of the chosen experts, as the grouped products take them: the entries
 * (t, j) with experts[t, j] in [first, first + G), in the order of (expert, t, j).
 * Others (experts of other GPUs, -1) are left out.
 *
 * offsets      out, int32 [G + 1]: rows offsets[g] .. offsets[g + 1] - 1 belong to expert
 *              first + g; offsets[0] = 0.
 * row_index    out, int32 [T * k]: the token of each row; 0 behind the last segment.
 * positions    out, int32 [T, k]: the row of each entry, -1 for those left out.
 * workspace    fp8fg_expert_segments_workspace(T, k, G) bytes, 4-byte aligned (0 bytes
 *              for few entries: NULL is fine then).
 * Requires 1 <= G <= 1024, first >= 0, first + G < 2^31, T * k < 2^31 - 2^20; 4-byte
 * alignment.  T == 0 or k == 0: offsets are set to zero.
 */
int fp8fg_expert_segments(const int32_t* experts, int64_t T, int64_t k, int64_t first, int64_t G, int32_t* offsets,
                          int32_t* row_index, int32_t* positions, void* workspace, int64_t workspace_bytes,
                          fp8fg_stream_t stream);
int64_t fp8fg_expert_segments_workspace(int64_t T, int64_t k, int64_t G);

/*
 * Combination of the experts' rows:  y[t] = base[t] + sum_j weights[t, j] * rows[positions[t, j]],
 * summed in fp32 in the order of j, rounded once.
 * With weights NULL (ones) and the rows' gradients it is the gradient of the dispatch.
 *
 * rows         [R, H] of `dtype`, row pitch ld_rows >= H.
 * positions    int32 [T, k]; values outside [0, R) add nothing.
 * weights      fp32 [T, k], or NULL.
 * base         [T, H] of `dtype`, row pitch ld_base >= H (a shared expert's output, the
 *              residual stream), or NULL.
 * y            out, [T, H] of `dtype`.
 * Requires H % 8 == 0, R < 2^31, T < 2^31, 0 <= k <= 32; rows, base, y 16-byte aligned,
 * ld * sizeof(elem) % 16 == 0, others 4-byte.  T == 0 or H == 0 is a no-op.
 */
int fp8fg_combine_experts(const void* rows, int dtype, int64_t R, int64_t H, int64_t ld_rows,
                          const int32_t* positions, const float* weights, int64_t T, int64_t k, const void* base,
                          int64_t ld_base, void* y, fp8fg_stream_t stream);

/*
 * Its gradient:  drows[positions[t, j]] = weights[t, j] * dy[t],
 *                dweights[t, j] = sum over the row of dy[t] * rows[positions[t, j]]   (fp32).
 * (base gets dy itself.)
 *
 * dy           [T, H] of `dtype`, row pitch ld_dy >= H.
 * rows         [R, H] of `dtype`, row pitch ld_rows >= H; may be NULL with dweights NULL.
 * positions    int32 [T, k], each row at most once, as fp8fg_expert_segments writes them
 *              (of a row that occurs twice either gradient may stay); values outside
 *              [0, R) write nothing, and 0 into dweights.
 * weights      fp32 [T, k], or NULL (ones).
 * drows        out, [R, H] of `dtype`, or NULL.  Rows that no position names stay as they
 *              were.
 * dweights     out, fp32 [T, k], or NULL.  One of both has to be asked for; where R == 0 or H == 0,
 *              rows and drows have no elements and are not looked at (dweights are 0).
 * Requirements as the forward call's.
 */
int fp8fg_combine_experts_backward(const void* dy, const void* rows, int dtype, int64_t R, int64_t H, int64_t ld_dy,
                                   int64_t ld_rows, const int32_t* positions, const float* weights, int64_t T,
                                   int64_t k, void* drows, float* dweights, fp8fg_stream_t stream);

/*
 * The same with the rows' gradient leaving 1x128-quantised (rule of fp8_quant_act_1x128,
 * or of its _pow2 form with pow2 == 1), for the data gradient of the experts' products.
 * A group whose largest value lies below 448 * 2^-126 gives zero codes, or with pow2
 * codes at the smallest normal scale.
 * q, scales    out, codes [R, H] (16-byte aligned) and fp32 [R, H/128].
 * Requires H % 128 == 0.
 */
int fp8fg_combine_experts_backward_quant(const void* dy, const void* rows, int dtype, int64_t R, int64_t H,
                                         int64_t ld_dy, int64_t ld_rows, const int32_t* positions,
                                         const float* weights, int64_t T, int64_t k, int pow2, uint8_t* q,
                                         float* scales, float* dweights, fp8fg_stream_t stream);

/*
 * 4-bit quantisation of a weight, groups of 32 along K (the OCP microscaling layout):
 *     per group  s = 2^e, e the smallest integer >= -126 with max|w| <= 6 * 2^e,
 *                code = E2M1_RNE(w * 2^-e)   (sign of w kept)
 * E2M1 codes: a sign bit over 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *
 * w            [N, K] of `w_dtype`, row pitch ld_w >= K elements; finite.
 * q            out, uint8 [N, K/2]: element 2i of a row in the low half of byte i, 2i + 1 in
 *              the high half.
 * scales       out, uint8 [N, K/32]: E8M0, the byte e + 127 (1 to 253).
 * Requires K % 128 == 0, N * K / 8 < 2^32 - 256; w 16-byte aligned, ld_w * sizeof(elem) %
 * 16 == 0, q 16-byte aligned, scales 4-byte.  N == 0 is a no-op.
 */
int fp4_quant_weight_1x32(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ld_w, uint8_t* q, uint8_t* scales,
                          fp8fg_stream_t stream);

/*
 * Products of few rows with 4-bit weights:  Y = X * deq(W)^T, every product exact, summed
 * in fp32.  The weights are read once per 32 rows of X, so this is for the rows of single
 * tokens; any number of rows is correct.
 *
 * x, sx        sx == NULL: X is bf16 [M, K].  Else E4M3 codes [M, K] and fp32 scales
 *              [M, K/128], as the 1x128 quantisers write them.
 * w, sw        codes [N, K/2] and scales [N, K/32] as fp4_quant_weight_1x32 writes them
 *              (scale bytes 0 and 255 give unspecified values, never a fault).
 * y            out, [M, N] of `y_dtype`.
 * Requires K % 128 == 0, 128 <= K < 2^24, M < 2^31, N < 2^31 (any N), (M + 1) * (N + 8) <
 * 2^35; x and w 16-byte aligned, sx, sw and y 4-byte (bf16 y 2-byte).  M == 0 or N == 0 is
 * a no-op.
 */
int fp4_gemm(const void* x, const float* sx, const uint8_t* w, const uint8_t* sw, void* y, int y_dtype, int64_t M,
             int64_t N, int64_t K, fp8fg_stream_t stream);

/*
 * The gated pair h = g * sigmoid(g) * u in one kernel: w [2I, K/2] and sw [2I, K/32] hold
 * the I gate rows, then the I up rows; h [M, I] of `h_dtype`.  Requires (I + 128) * K <
 * 2^33; otherwise as fp4_gemm.
 */
int fp4_gated_gemm(const void* x, const float* sx, const uint8_t* w, const uint8_t* sw, void* h, int h_dtype,
                   int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream);

/*
 * Both over expert row segments (offsets, rows as fp8_block_grouped_gemm_gather, or as
 * fp8fg_expert_segments writes them): row r of segment e takes token row_index[r], or row
 * r of X when row_index is NULL (then T must equal M_total).
 * w, sw        codes [G, N, K/2] and scales [G, N, K/32]  (gated: N = 2I).
 * y, h         out, [M_total, N] or [M_total, I], in routed-row order.  Rows behind
 *              group_offsets[G] stay as they were.
 * Offsets below 0 or above M_total, and indices outside [0, T), are held to these; with
 * offsets that decrease nothing is written.  Never an access outside the operands.
 * Requires G < 2^31, (M_total + 2 * min(G, M_total)) * (N + 8) < 2^35, and with row_index an X of
 * less than 4 GiB; otherwise as above.
 */
int fp4_grouped_gemm(const void* x, const float* sx, int64_t T, const int32_t* row_index,
                     const int32_t* group_offsets, int64_t G, const uint8_t* w, const uint8_t* sw, void* y,
                     int y_dtype, int64_t M_total, int64_t N, int64_t K, fp8fg_stream_t stream);
int fp4_grouped_gated_gemm(const void* x, const float* sx, int64_t T, const int32_t* row_index,
                           const int32_t* group_offsets, int64_t G, const uint8_t* w, const uint8_t* sw, void* h,
                           int h_dtype, int64_t M_total, int64_t I, int64_t K, fp8fg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_EXPERTS_H */
