/*
 * libmxmoe, training step of unquantized experts -- products grouped by
 * expert on bf16 operands with their gradients, the global norm of many
 * gradient tensors, and the AdamW step over many tensors at once with its
 * states in 32 or in 8 bits.  C ABI, same library and same conventions as
 * libmxmoe.h (device pointers owned by the caller, nothing allocated, no
 * synchronization, host-checkable preconditions validated before any launch,
 * group_offsets int32 [G+1] on the device and clamped there to [0, M]).
 *
 * A mixed-precision recipe keeps some expert layers out of MXFP8 (typically
 * the first and last ones) and needs an optimizer for all of them: the
 * weight gradients written here, or by mx_grouped_gemm_wgrad, are what
 * mx_grad_norm and mx_adamw read, and the bf16 weights that mx_adamw writes
 * are what these products, or mx_quantize_dual, read in the next step.
 */
#ifndef LIBMXMOE_TRAIN_H
#define LIBMXMOE_TRAIN_H
#include "libmxmoe.h"
#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward product: out[r][n] = sum_k x[r][k] w[g][n][k] for the rows r of
 * group g, accumulated in fp32 and rounded to bf16 once.  Rows outside every
 * group are left alone.
 *   x    bf16 [M][ldx] (first K columns used)
 *   w    bf16 [G][N][K], contiguous
 *   out  bf16 [M][ldo] (first N columns written)
 * Requires N % 8 == 0, K % 8 == 0, ldx >= K, ldo >= N (MX_ERR_SHAPE);
 * 16-byte aligned pointers, ldx % 8 == 0, ldo % 8 == 0 (MX_ERR_ALIGN).
 * K = 0 writes zeros.  MX_ERR_UNSUPPORTED from N, K or a row stride of 2^22
 * elements, from N K = 2^31, or from M = 2^31 on.
 */
mx_status mx_grouped_gemm_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* group_offsets,
                               int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldo, void* stream);

/*
 * Input gradient: dx[r][k] = sum_n dy[r][n] w[g][n][k] for the rows r of
 * group g; w is read as the forward product reads it (no transposed copy).
 *   dy   bf16 [M][ldy] (first N columns used)
 *   w    bf16 [G][N][K], contiguous
 *   dx   bf16 [M][ldx] (first K columns written)
 * Requirements as above, with the roles of N and K as named here; N = 0
 * writes zeros.
 */
mx_status mx_grouped_gemm_bf16_dgrad(const uint16_t* dy, int64_t ldy, const uint16_t* w, const int32_t* group_offsets,
                                     int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* dx, int64_t ldx,
                                     void* stream);

/*
 * Weight gradient: dw[g][n][k] = sum over the rows r of group g of
 * dy[r][n] x[r][k], accumulated in fp32.
 *   dy   bf16 [M][ldy] (first N columns used), x bf16 [M][ldx] (first K)
 *   dw   [G][N][K], contiguous: bf16 (dw_fp32 = 0, rounded once) or fp32
 *        (dw_fp32 = 1); with accumulate = 1 the product is added to the fp32
 *        values already there (MX_ERR_UNSUPPORTED for a bf16 dw: repeated
 *        rounding would lose the small ones).
 * A group without rows gives zeros (with accumulate: no change).
 *   workspace  scratch memory of workspace_bytes, 16-byte aligned, or NULL: few
 *        weights and long groups leave most of the GPU idle unless the rows
 *        of a group are shared out and the parts' sums (fp32, kept here)
 *        joined.  It is used if it has mx_grouped_gemm_bf16_wgrad_workspace_bytes
 *        (0 where nothing would be shared out, -1 for invalid sizes); the
 *        result differs by fp32 roundings.
 * Requirements as above; dw_fp32 and accumulate are 0 or 1 and
 * workspace_bytes >= 0 (MX_ERR_SHAPE).
 */
mx_status mx_grouped_gemm_bf16_wgrad(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                     const int32_t* group_offsets, int32_t G, int64_t M, int64_t N, int64_t K,
                                     void* dw, int32_t dw_fp32, int32_t accumulate, void* workspace,
                                     int64_t workspace_bytes, void* stream);
int64_t mx_grouped_gemm_bf16_wgrad_workspace_bytes(int32_t G, int64_t M, int64_t N, int64_t K);

/* Types of a tensor of the optimizer (mx_adamw_tensor.types). */
enum {
    MX_ADAMW_W_BF16 = 1,     /* w is bf16 (else float32) */
    MX_ADAMW_G_BF16 = 2,     /* g is bf16 (else float32) */
    MX_ADAMW_STATE_8BIT = 4, /* m and v are E4M3 codes with block scales (else float32) */
    MX_ADAMW_UNBIASED = 16   /* their codes are rounded at random, without bias (else to nearest) */
};

/* Elements per scale of an 8-bit state. */
#define MX_ADAMW_BLOCK 256

/*
 * One tensor of n elements (device pointers, each aligned to its element).
 *   w        weights, written by the step
 *   master   float32 [n]: the values that w rounds, or NULL.  With it the step
 *            updates master and writes its rounding to w (which it does not
 *            read); without it w itself is updated.  Only with MX_ADAMW_W_BF16.
 *   g        gradients, read
 *   m, v     states, updated
 *   m_scale, v_scale   float32 [ceil(n / 256)], 8-bit states only (else NULL)
 * An 8-bit state: block b holds elements [256 b, 256 b + 256).  m = m_scale[b]
 * code(m), v = (v_scale[b] code(v))^2, codes OCP E4M3FN (v: not negative).
 * Zero codes and scales are the state before the first step.
 *
 * Codes rounded to nearest hold their state for what a step changes by less
 * than half a code's step: sqrt(v) falls by no more than 1 - sqrt(beta2) a
 * step, so the code of an element that is not its block's largest stays for as
 * long as the block's largest stays, whatever its own gradients do.  (Where one
 * element of a block keeps its gradient and the others' fall to a hundredth,
 * their v stays 10^4 times too large; with Gaussian gradients v is 15 % too
 * large on average at beta2 = 0.95 and 24 % at 0.999.)  For training, set
 * MX_ADAMW_UNBIASED: m and v are then right on average over the roundings.
 */
typedef struct {
    void* w;
    float* master;
    const void* g;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int64_t n;
    float weight_decay;
    uint32_t types;
} mx_adamw_tensor;

/*
 * The plan of a list of tensors: what the two calls below read on the device
 * to share the work out.  mx_adamw_plan checks the list (host memory) and
 * writes the plan to `plan` (host memory of mx_adamw_plan_bytes bytes); the
 * caller copies it to the device once (16-byte aligned) and keeps it while
 * the tensors stay where they are.  *chunks receives a number that those
 * calls take.
 * MX_ERR_NULL: a required pointer is NULL (m_scale and v_scale are required
 * for 8-bit states); MX_ERR_SHAPE: count < 0, n < 0, unknown type bits, a
 * master with float32 weights, a weight decay that is negative or not
 * finite, scales or unbiased codes with 32-bit states; MX_ERR_ALIGN: a pointer is not aligned
 * to its element; MX_ERR_UNSUPPORTED: more than 2^31 - 1 chunks.
 * mx_adamw_plan_bytes returns -1 for a list that mx_adamw_plan rejects for
 * its count or a length.
 */
int64_t mx_adamw_plan_bytes(const mx_adamw_tensor* tensors, int32_t count);
mx_status mx_adamw_plan(const mx_adamw_tensor* tensors, int32_t count, void* plan, int64_t* chunks);

/* Bytes of the workspace of mx_grad_norm (zeroed once by the caller before
 * its first use; one call at a time may use it). */
int64_t mx_grad_norm_workspace_bytes(void);

/*
 * Global norm of the gradients of a plan, and the factor that clips them:
 *   out[0] = sqrt(sum g^2) over all tensors
 *   out[1] = min(1, max_norm / out[0]); NaN if the norm is not finite
 * Squares are summed in double in an order that depends on the plan only
 * (the same input gives the same bits).  max_norm > 0, infinity = no
 * clipping (MX_ERR_SHAPE otherwise).  out: float32 [2] on the device.
 */
mx_status mx_grad_norm(const void* plan, int32_t count, int64_t chunks, float max_norm, void* workspace, float* out,
                       void* stream);

/*
 * One AdamW step of every tensor of a plan.  With t = the step count after
 * this step, c = *grad_scale (1 if NULL) and per element, in fp32,
 *   g' = c g
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   w  = keep w - size (m / (sqrt(v) root + eps))
 * with keep = 1 - lr decay, size = lr / (1 - beta1^t), root = 1 / sqrt(1 -
 * beta2^t), each formed in double and rounded to fp32 once.
 * The new w uses m and v before they are rounded to 8 bits:
 *   scale = max(amax, 2^-100) / 448 over the block of 256, code = E4M3(x / scale)
 * with x = m, or x = sqrt(v), to nearest even; the code of a v > 0 is at
 * least the smallest one, 2^-9, so that no later step divides by eps alone
 * (below sqrt(v) = 2^-57 the code's square can underflow: there it does).
 * Tensors with MX_ADAMW_UNBIASED take one of the two codes next to x / scale,
 * at random: m's with the expected value x / scale, v's with the expected
 * square (x / scale)^2 (but for that smallest code).  The random numbers depend
 * on t and the element's index in its tensor only, so that the same step gives
 * the same bits, in whatever list its tensor stands.
 * Every operation is rounded to fp32 by itself, in the order that the
 * parentheses give; x / scale is x times ((1 / amax) times 448), the scale amax
 * times 1/448.
 *   steps       int64 [2] on the device: [0] the number of steps done, which
 *               the call raises by one; [1] zero, used by the call
 *   lr, lr_device   the learning rate, or (not NULL) a float32 on the device
 *               to take in its place, for captured graphs with a schedule
 *               (taken as it is: one that is not finite reaches the weights)
 *   grad_scale  float32 on the device or NULL.  If it is negative or not
 *               finite, the call changes nothing (out + 1 of mx_grad_norm:
 *               a step with infinite or NaN gradients is left out)
 * Without such a factor a NaN or infinity in g reaches m, v and w of its
 * element and, with 8-bit states, the states of its block.
 * MX_ERR_SHAPE unless 0 <= beta1 < 1, 0 <= beta2 < 1, eps >= 0 and lr are
 * finite and count and chunks not negative (with eps = 0 a weight whose v is
 * 0 becomes NaN, as the formula has it).  count, chunks: the plan's; an empty
 * plan still counts the step.
 */
mx_status mx_adamw(const void* plan, int32_t count, int64_t chunks, int64_t* steps, double lr, const float* lr_device,
                   double beta1, double beta2, double eps, const float* grad_scale, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LIBMXMOE_TRAIN_H */
