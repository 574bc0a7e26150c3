/*
 * fp8fg_layer -- the operators between the FP8 GEMMs of a feed-forward sublayer
 * (training step and single-token serving), on gfx950.
 *
 * Same library, status codes, element types and conventions as fp8fg.h: device
 * pointers unless stated otherwise, nothing allocated or retained, no
 * synchronisation, every argument checked on the host before anything is
 * enqueued, no exception across the boundary, capturable in a HIP graph.
 * Workspaces are the caller's; a call's workspace may be reused once the stream
 * has passed the call.  Outputs must not alias inputs unless stated otherwise.
 */
#ifndef FP8FG_LAYER_H
#define FP8FG_LAYER_H

#include "fp8fg.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition, root-mean-square norm and 1x128 quantisation, one pass:
 *     z = x + residual                                (fp32)
 *     rstd = 1 / sqrt(mean(z^2) + eps),  y = z * rstd * weight
 *     q, scales = the 1x128 quantisation of y (rule of fp8_quant_act_1x128, or of
 *                 fp8_quant_act_1x128_pow2 with pow2 == 1)
 *     h = z rounded to `dtype`, for the residual stream and the backward pass.
 * y comes from the unrounded z.  z^2 is summed in fp32, so |z| beyond about 1e19
 * is outside the range; other finite inputs are fine.  A row of zeros gives zero
 * codes and scales.  With eps == 0 rstd has its full precision where mean(z^2) is
 * at least 2^-126, and a row whose mean(z^2) is zero in fp32 (zeros, or |z| below
 * about 1e-22) counts as a row of zeros, with rstd = 0.  A group whose largest |y|
 * lies below 448 * 2^-126 gives zero codes, or with pow2 codes at the smallest
 * normal scale.
 *
 * x, residual  [M, H] of `dtype`, row pitches ld_x, ld_r >= H elements; residual
 *              may be NULL (then z = x).
 * weight       [H] of `w_dtype`.
 * h            out [M, H] of `dtype`, or NULL.
 * y            out [M, H] of `dtype` (y in high precision), or NULL.
 * q, scales    out, codes [M, H] and fp32 [M, H/128].
 * rstd         out, fp32 [M], or NULL.
 * Requires H % 128 == 0 and H <= 32768; x, residual, weight, h, y and q 16-byte
 * aligned, ld * sizeof(elem) % 16 == 0, scales and rstd 4-byte aligned; eps >= 0.
 * M == 0 is a no-op.
 */
int fp8_add_rmsnorm_quant_1x128(const void* x, const void* residual, int dtype, int64_t M, int64_t H, int64_t ld_x,
                                int64_t ld_r, const void* weight, int w_dtype, float eps, int pow2, void* h, void* y,
                                uint8_t* q, float* scales, float* rstd, fp8fg_stream_t stream);

/*
 * Gradient of the norm (the quantisation passes gradients through unchanged):
 * with n = h * rstd and d = dy * weight,
 *     dx = rstd * (d - n * mean(d * n)) + dh,   dw = sum over rows of dy * n.
 * dx is the gradient of both x and the residual.  A row with rstd == 0 (see the
 * forward call) has dx = dh and adds nothing to dw.  dw is summed in fp32, in an
 * order fixed by M and H alone: the same bits on every run.
 *
 * dy, h, dh    [M, H] of `dtype`, row pitches ld_* >= H; dh, the gradient that
 *              arrives along the residual stream, may be NULL (zero).
 * rstd         fp32 [M], as the forward call wrote it.
 * weight       [H] of `w_dtype`.
 * dx           out [M, H] of `dtype`.
 * dw           out, fp32 [H], or NULL (then no workspace is needed).  Zero if M == 0.
 * workspace    fp8_rmsnorm_backward_workspace(M, H) bytes, 16-byte aligned.
 * Requirements as the forward call's.
 */
int fp8_rmsnorm_backward(const void* dy, const void* h, const void* dh, int dtype, int64_t M, int64_t H, int64_t ld_dy,
                         int64_t ld_h, int64_t ld_dh, const float* rstd, const void* weight, int w_dtype, void* dx,
                         float* dw, void* workspace, int64_t workspace_bytes, fp8fg_stream_t stream);
int64_t fp8_rmsnorm_backward_workspace(int64_t M, int64_t H);

/*
 * Gated pair of block-scaled FP8 products, with the activation and the product
 * in the same kernel (the gate and up projections of a feed-forward block):
 *     g = deq(A) deq(W[0:I])^T,  u = deq(A) deq(W[I:2I])^T    (fp8_block_gemm's sums)
 *     h = g * sigmoid(g) * u                                  (fp32)
 *
 * a, sa        codes [M, K] and scales [M, K/128] (1x128).
 * w, sw        codes [2I, K], gate rows first, and scales [2I/128, K/128]
 *              (128x128): the quantisation of the two weights stacked.
 * accum        FP8FG_ACCUM_FP8_MFMA, FP8FG_ACCUM_EXACT or FP8FG_ACCUM_SCALED_MFMA.
 * h            out [M, I] of `h_dtype`.
 * gu           out [M, 2I] of `h_dtype`, g then u, for the backward pass; or NULL.
 * Requires K % 128 == 0 with 128 <= K < 2^24, I % 128 == 0, at most 8388600 tiles of
 * 128 x 128 outputs (ceil(M / 128) * I / 128; over experts (M_total / 128 + G) *
 * I / 128); a, w, h, gu 16-byte aligned, scales 4-byte.  M == 0 or I == 0 is a no-op.
 */
int fp8_block_gated_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum, void* h,
                         int h_dtype, void* gu, int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream);

/*
 * The same with h leaving 1x128-quantised along I (rule of fp8_quant_act_1x128, or
 * of fp8_quant_act_1x128_pow2 with pow2 == 1), ready for the down projection.  A
 * group whose largest |h| lies below 448 * 2^-126 gives zero codes, or with pow2
 * codes at the smallest normal scale.
 * q_h, s_h     out, codes [M, I] (16-byte aligned) and fp32 [M, I/128].
 * gu           out, bf16 [M, 2I], or NULL.
 * workspace    4 * M * I bytes, 16-byte aligned, or NULL.  With few rows the work is
 *              spread over small tiles that hold no whole group: h then passes
 *              through the workspace in fp32 and a second kernel quantises it.
 *              Without one (or with a smaller one) one kernel does it all, several
 *              times slower there.
 * fp8_block_gated_gemm_quant_workspace: the bytes a call with these sizes would
 * use, 0 for none (G: experts of the grouped form, 0 for the dense one).
 */
int fp8_block_gated_gemm_quant(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum,
                               int pow2, uint8_t* q_h, float* s_h, void* gu, void* workspace, int64_t workspace_bytes,
                               int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream);
int64_t fp8_block_gated_gemm_quant_workspace(int accum, int64_t M, int64_t I, int64_t K, int64_t G);

/*
 * The gated pair over expert row segments (offsets, rows and weights as
 * fp8_block_grouped_gemm_gather): row r of segment e takes token row_index[r],
 * or row r of A when row_index is NULL (then T must equal M_total).
 * w, sw        codes [G, 2I, K] and scales [G, 2I/128, K/128].
 * h, gu        out [M_total, I] and [M_total, 2I] (or NULL), in routed-row order.
 * Requires T * K < 2^32; otherwise as the calls above and the grouped GEMM.
 */
int fp8_block_grouped_gated_gemm(const uint8_t* a, const float* sa, int64_t T, const int32_t* row_index,
                                 const int32_t* group_offsets, int64_t G, const uint8_t* w, const float* sw,
                                 int accum, void* h, int h_dtype, void* gu, int64_t M_total, int64_t I, int64_t K,
                                 fp8fg_stream_t stream);
int fp8_block_grouped_gated_gemm_quant(const uint8_t* a, const float* sa, int64_t T, const int32_t* row_index,
                                       const int32_t* group_offsets, int64_t G, const uint8_t* w, const float* sw,
                                       int accum, int pow2, uint8_t* q_h, float* s_h, void* gu, void* workspace,
                                       int64_t workspace_bytes, int64_t M_total, int64_t I, int64_t K,
                                       fp8fg_stream_t stream);

/*
 * Gradient of the gated activation, quantised as it is formed.  With g, u the
 * halves of gu and p = sigmoid(g) (fp32):
 *     dg = dh u p (1 + g (1 - p)),   du = dh g p,   h = g p u
 *     q, s        [M, 2I], [M, 2I/128]: (dg, du) 1x128-quantised along its columns;
 *                 dX = fp8_block_gemm of it with the transposed weight codes of
 *                 fp8_quant_weight_128x128_dual.
 *     q_t, s_t    [2I, M], [2I, M/128]: its transpose, quantised along the tokens;
 *                 dW of the gate and up weights = fp8_block_gemm (FP8FG_B_ROW_1x128)
 *                 of it with the transposed quantisation of X.
 *     q_ht, s_ht  [I, M], [I, M/128]: h transposed, quantised along the tokens, for
 *                 the down projection's dW.
 * The groups along the tokens start at row 0, whatever experts the rows belong to: for
 * the weight gradients of experts, one call per expert on its rows, zero rows added
 * to a multiple of 128.
 * Quantisation by the rule of fp8_quant_act_1x128, or of its _pow2 form; a group whose
 * largest value lies below 448 * 2^-126 (saturated gates, say) has zero codes, or with
 * pow2 codes at the smallest normal scale.
 *
 * dh           [M, I] of `dtype`, row pitch ld_dh >= I.
 * gu           [M, 2I] of `dtype`, as the forward call saved it.
 * Each output pair may be NULL (both of it), but not all three.
 * Requires I % 128 == 0, and M % 128 == 0 for the transposed pairs; M * I / 128 at
 * most 2^31 - 9, for q alone 2^28 - 16, for transposed pairs of fp32 values 2^30 -
 * 1024; dh, gu, q, q_t and q_ht 16-byte aligned, ld_dh * sizeof(elem) % 16 == 0,
 * scales 4-byte.
 * M == 0 or I == 0 is a no-op.
 */
int fp8_gated_backward_quant(const void* dh, const void* gu, int dtype, int64_t M, int64_t I, int64_t ld_dh, int pow2,
                             uint8_t* q, float* s, uint8_t* q_t, float* s_t, uint8_t* q_ht, float* s_ht,
                             fp8fg_stream_t stream);

/*
 * Global norm over n gradients:  norm = sqrt(sum of squares over all of them),
 * squares summed in 64 bits, in an order fixed by the lengths alone.
 *
 * grads, counts, dtypes   HOST arrays of n device pointers, element counts (>= 0)
 *              and element types; read during the call only.  A tensor of count
 *              0 may have a null pointer.  Pointers need their element's alignment.
 * norm         out, fp32 [1] (device).  Zero for n == 0.
 * workspace    fp8fg_grad_norm_workspace(n) bytes, 8-byte aligned.
 */
int fp8fg_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t n, float* norm,
                    void* workspace, int64_t workspace_bytes, fp8fg_stream_t stream);

/*
 * The same norm, and every gradient scaled by
 *     c = norm <= max_norm ? 1 : max_norm / norm
 * (a norm that is not a number makes c, and so every output, not a number).
 * outs         HOST array of n device pointers, of the gradients' types and
 *              counts; outs[i] == grads[i] scales in place.  No output may
 *              overlap another output or another gradient, or its own in part
 *              (FP8FG_ERR_INVALID_ARG): a tensor listed twice would be scaled
 *              while it is read.  fp8fg_grad_norm takes any list.
 * Requires max_norm > 0.  Other arguments as fp8fg_grad_norm.
 */
int fp8fg_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes,
                         int64_t n, float max_norm, float* norm, void* workspace, int64_t workspace_bytes,
                         fp8fg_stream_t stream);
int64_t fp8fg_grad_norm_workspace(int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_LAYER_H */
