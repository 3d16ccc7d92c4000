/*
 * libmxmoe, what surrounds the experts in a block of a mixture-of-experts
 * model -- the router (from logits to experts and weights) with its gradient,
 * the gradient of the routing weights through the combine, and the
 * root-mean-square norm in front of the block, with the residual's addition
 * and an MXFP8 copy of its output, with its gradient.  C ABI, same library
 * and same conventions as libmxmoe.h (device pointers owned by the caller,
 * nothing allocated, no synchronization, host-checkable preconditions
 * validated before any launch).
 *
 * mx_router writes the experts and weights that mx_route_plan and mx_combine
 * take; mx_combine_dweights and mx_router_backward lead the output gradient
 * back to the logits; mx_rms_norm writes the bf16 rows that the router's
 * product and mx_gather_quantize read, and the MXFP8 rows that
 * mx_grouped_gemm and mx_grouped_gemm_swiglu read as X.
 */
#ifndef LIBMXMOE_BLOCK_H
#define LIBMXMOE_BLOCK_H
#include "libmxmoe.h"
#ifdef __cplusplus
extern "C" {
#endif

/* Flags of the router's calls. */
enum {
    MX_ROUTER_SIGMOID = 1,    /* scores are sigmoids of the logits (else their softmax) */
    MX_ROUTER_RENORM = 2,     /* weights are divided by their sum over the experts chosen */
    MX_ROUTER_LOGITS_BF16 = 4 /* logits (and their gradient) are bf16 (else float32) */
};

/* Experts chosen per token, and groups of experts, at most. */
#define MX_ROUTER_MAX_K 64
#define MX_ROUTER_MAX_GROUPS 64

/*
 * Router: for each token t with logits l[e], e < E,
 *   s[e] = e^l[e] / sum e^l, or 1 / (1 + e^-l[e])      the scores
 *   c[e] = s[e] + bias[e] (c = s without a bias)        the choices
 * An expert whose logit or bias is -infinity (a mask) is never chosen.
 * With groups > 1 the experts form groups of E / groups consecutive ones; a
 * group's score is the sum of its group_top largest choices (of one, if only
 * one expert of it can be chosen), and only experts of the groups_kept groups
 * of the largest scores can be chosen.  Then
 *   experts[t][i], i < k: the k largest choices, largest first
 *   weights[t][i] = scale s[e_i], divided by sum_j s[e_j] with RENORM (0
 *                   where that sum is 0)
 * and -1 with weight 0 for the choices that too few experts are left for (a
 * token whose mask leaves nothing has only those; mx_route_plan drops them).
 * Ties go to the lower index, for experts and groups.  The bias decides who is
 * chosen and is not part of the weights.
 *   logits   float32 or bf16 [T][ldl] (first E columns used)
 *   bias     NULL, or float32 [E]
 *   experts  int32 [T][k] out; weights float32 [T][k] out
 *   scores   NULL, or float32 [T][E] out: all scores (of masked experts too;
 *            zeros for a token whose logits are all -infinity)
 * Outputs overlap nothing else: logits are read again after scores are written
 * (scores in the place of logits: MX_ERR_SHAPE).
 * Choices are compared in binary64, so that ones that binary32 cannot tell
 * apart are in the order of the formulas (without a bias, and with one choice
 * per group score, the logits themselves are compared: the order is the same).
 * Weights are formed in binary64 and rounded once, but for the softmax's sum
 * over all experts, which is of binary32 (weights without RENORM: a few
 * steps), as the scores output is.  A token's results do not depend on the
 * others', only on the sizes.
 * A NaN, in a logit or choice, counts as larger than every number; that of a
 * logit makes its weight NaN (with RENORM or the softmax all of the token's).
 * Requires T >= 0, 1 <= E <= 4096, 1 <= k <= 64, 1 <= groups <= 64, E %
 * groups == 0, 1 <= groups_kept <= groups, k <= groups_kept E / groups,
 * group_top 1 or 2, ldl >= E, finite scale (MX_ERR_SHAPE); pointers aligned to
 * their elements (MX_ERR_ALIGN); T < 2^24, and for a number of groups that is
 * no power of two E p / groups <= 4096 with p the next one; strides < 2^32
 * (MX_ERR_UNSUPPORTED).
 */
mx_status mx_router(const void* logits, int64_t ldl, int64_t T, int32_t E, const float* bias, int32_t groups,
                    int32_t groups_kept, int32_t group_top, int32_t k, float scale, uint32_t flags, int32_t* experts,
                    float* weights, float* scores, void* stream);

/*
 * Gradient of the logits: with g[i] = dweights[t][i] and the chosen experts
 * e_i (entries outside [0, E) are left out; an expert that is named twice
 * counts twice),
 *   ds[e] = dscores[t][e] + sum over i with e_i = e of
 *           scale (g[i] - sum_j g[j] s[e_j] / S) / S,  S = sum_j s[e_j], with
 *           RENORM (0 where S is 0), and of scale g[i] without
 *   dl[e] = s[e] (ds[e] - sum_f s[f] ds[f])   softmax
 *   dl[e] = s[e] (1 - s[e]) ds[e]             sigmoid
 * in fp32, rounded to the type of the logits once.  With RENORM the ratios
 * s[e_i] / S are formed from differences of the chosen logits, so that scores
 * need not be numbers of binary32; S counts as 0 where mx_router's does with
 * the sigmoid (every chosen logit is below -709.78), and never with the
 * softmax (there too the gradient is that of the ratios).  The choice itself
 * has no gradient, and the bias none.
 *   logits    as mx_router; experts int32 [T][k], dweights float32 [T][k]
 *   dscores   NULL, or float32 [T][E]: a gradient of the scores output
 *   dlogits   float32 or bf16, as the logits, [T][ldd] out (E columns
 *             written); may be logits themselves (same stride)
 * Logits of -infinity get 0.  Requirements as above.
 */
mx_status mx_router_backward(const void* logits, int64_t ldl, int64_t T, int32_t E, const int32_t* experts,
                             const float* dweights, const float* dscores, int32_t k, float scale, uint32_t flags,
                             void* dlogits, int64_t ldd, void* stream);

/*
 * Gradient of the weights of mx_combine:
 *   dweights[t][i] = sum_n dout[t][n] y[slot_of[t][i]][n]
 * in fp32, in an order that depends on the sizes only (the same input gives
 * the same bits); 0 for entries whose slot lies outside [0, M).
 *   dout     bf16 [T][ldd] (first N columns used)
 *   y        bf16 [M][ldy] expert-ordered rows (may be NULL when M == 0)
 *   slot_of  int32 [T][k] (mx_route_plan)
 *   dweights float32 [T][k] out
 * Requires N % 8 == 0 (MX_ERR_UNSUPPORTED), ldd, ldy >= N, k >= 1
 * (MX_ERR_SHAPE), dout, y 16-byte aligned, ldd, ldy % 8 == 0, slot_of and
 * dweights 4-byte aligned (MX_ERR_ALIGN); T < 2^24, M and T k < 2^31, ldd and
 * ldy < 2^30 (MX_ERR_UNSUPPORTED).
 */
mx_status mx_combine_dweights(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t M, int64_t ldy,
                              const int32_t* slot_of, int64_t T, int32_t k, int64_t N, float* dweights, void* stream);

/* Flags of the norm's calls. */
enum {
    MX_NORM_STREAM_FP32 = 1, /* the residual stream (residual, h, dh_in, dh) is float32 (else bf16) */
    MX_NORM_WEIGHT_FP32 = 2  /* the weight is float32 (else bf16) */
};

/* Longest row of the norm. */
#define MX_NORM_MAX_N 32768

/*
 * Root-mean-square norm of M rows of N columns, with the residual's addition
 * before it and an MXFP8 copy of its output:
 *   h = x + residual, rounded to the stream's type (h = x without a residual)
 *   r = 1 / sqrt(sum_n h[n]^2 / N + eps),   y[n] = bf16(h[n] r w[n])
 *   (q, s) = the output of mx_quantize_rows(y), byte for byte (padding too)
 * h is rounded before it is normed, so that y is the norm of the stream that
 * the next layer and the backward pass read; everything else is fp32 (r, the
 * products and sums), and y is rounded once.
 *   x         bf16 [M][ldx], or float32 for a float32 stream without a
 *             residual (then h = x)
 *   residual  NULL, or [M][ldr] of the stream's type
 *   weight    [N]
 *   h         NULL, or [M][ldh] of the stream's type: the sum.  Required with a
 *             residual (MX_ERR_NULL), not allowed without (MX_ERR_SHAPE)
 *   y         NULL, or bf16 [M][ldy]
 *   q, s      NULL both (one alone: MX_ERR_NULL), or codes uint8 [M][N] and
 *             packed scales (mx_scale_bytes(M, N)); N % 32 == 0 (MX_ERR_SHAPE)
 *   rstd      NULL, or float32 [M]: r, for the backward pass
 * h may be residual, and h or y may be x, where type and stride are the same;
 * outputs overlap nothing else.  N is at most 32768, M < 2^31
 * (MX_ERR_UNSUPPORTED).  Requires N % 8 == 0, N > 0, strides >= N, eps >= 0 and
 * finite (MX_ERR_SHAPE; with eps = 0 a row of zeros gives NaN, as the formula
 * has it), 16-byte aligned pointers (rstd, s: 4), strides that are multiples
 * of 8 (MX_ERR_ALIGN) and below 2^30 (MX_ERR_UNSUPPORTED).  Rows that are not
 * finite give y as the formula does and unspecified codes.
 */
mx_status mx_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, int64_t M,
                      int64_t N, float eps, uint32_t flags, void* h, int64_t ldh, uint16_t* y, int64_t ldy,
                      uint8_t* q, uint8_t* s, float* rstd, void* stream);

/*
 * Its gradients, from the h and rstd of the forward pass.  With g = dy (+ dy2,
 * in fp32), a = g w and z = h rstd per row,
 *   dh = dh_in + rstd (a - z sum_n a[n] z[n] / N),   dweight = sum over rows of g z
 * The gradient of the sum is that of both x and the residual.
 *   dy       bf16 [M][ldy]; dy2 NULL, or bf16 [M][ldy2]: a second gradient of y
 *            (its other reader's)
 *   h        [M][ldh] of the stream's type; rstd float32 [M]
 *   dh_in    NULL, or [M][ldi] of the stream's type: the gradient that reaches
 *            h from behind (the residual stream)
 *   dh       [M][ldo] of the stream's type, out
 *   dx       NULL, or bf16 [M][lddx] out: the value of dh rounded to bf16 (only
 *            for a float32 stream, MX_ERR_SHAPE: of a bf16 one dh is it)
 *            dh and dx may each be one of dy, dy2, h and dh_in, where type and
 *            stride are the same; outputs overlap nothing else
 *   dweight  NULL, or [N]: bf16 (dw_fp32 = 0) or float32 (dw_fp32 = 1); with
 *            accumulate = 1 the sum is added to the float32 values there
 *            (MX_ERR_UNSUPPORTED for bf16)
 *   workspace  scratch memory of mx_rms_norm_backward_workspace_bytes(M, N)
 *            (0 for few rows), 16-byte aligned, for dweight (MX_ERR_CAPACITY if
 *            smaller); calls on several streams need one each
 * dweight is summed in fp32 in an order that depends only on the sizes and, for
 * few rows, on whether an output replaces dy, dy2 or h.
 * M = 0 writes zeros to dweight (with accumulate: no change).  Requirements
 * as above, M < 2^31.  mx_rms_norm_backward_workspace_bytes returns -1 for
 * sizes that the call refuses.
 */
mx_status mx_rms_norm_backward(const uint16_t* dy, int64_t ldy, const uint16_t* dy2, int64_t ldy2, const void* h,
                               int64_t ldh, const void* weight, const float* rstd, const void* dh_in, int64_t ldi,
                               int64_t M, int64_t N, uint32_t flags, void* dh, int64_t ldo, uint16_t* dx, int64_t lddx,
                               void* dweight, int32_t dw_fp32, int32_t accumulate, void* workspace,
                               int64_t workspace_bytes, void* stream);
int64_t mx_rms_norm_backward_workspace_bytes(int64_t M, int64_t N);

#ifdef __cplusplus
}
#endif
#endif /* LIBMXMOE_BLOCK_H */
