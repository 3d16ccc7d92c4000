// C-ABI entry points of what surrounds the experts: argument validation, then
// the launchers.  See include/libmxmoe_block.h for the contract of each call.
#include "../../include/libmxmoe_block.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "mx_block.h"

namespace {

bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }

mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

constexpr int32_t kMaxExperts = 4096;
constexpr int64_t kMaxTokens = (int64_t)1 << 24;  // a team of up to 64 lanes each: the grid's limit
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 32;  // of a token: offsets in bytes stay far below 2^63

mx_status check_router(int64_t ldl, int64_t T, int32_t E, int32_t k, float scale, uint32_t flags) {
    if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > MX_ROUTER_MAX_K || ldl < E || !std::isfinite(scale))
        return MX_ERR_SHAPE;
    if ((flags & ~(uint32_t)(MX_ROUTER_SIGMOID | MX_ROUTER_RENORM | MX_ROUTER_LOGITS_BF16)) != 0) return MX_ERR_SHAPE;
    if (T >= kMaxTokens || ldl >= kMaxStride) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

mx_status check_norm(int64_t M, int64_t N, uint32_t flags) {
    if (M < 0 || N <= 0 || N % 8 != 0) return MX_ERR_SHAPE;
    if ((flags & ~(uint32_t)(MX_NORM_STREAM_FP32 | MX_NORM_WEIGHT_FP32)) != 0) return MX_ERR_SHAPE;
    if (M >= kMaxRows || N > MX_NORM_MAX_N) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

// A row stride: of a matrix that is there, or unused.
mx_status check_stride(const void* p, int64_t ld, int64_t N) {
    if (!p) return MX_OK;
    if (ld < N) return MX_ERR_SHAPE;
    if (ld % 8 != 0) return MX_ERR_ALIGN;
    return ld >= (int64_t)1 << 30 ? MX_ERR_UNSUPPORTED : MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_router(const void* logits, int64_t ldl, int64_t T, int32_t E, const float* bias, int32_t groups,
                    int32_t groups_kept, int32_t group_top, int32_t k, float scale, uint32_t flags, int32_t* experts,
                    float* weights, float* scores, void* stream) {
    const mx_status st = check_router(ldl, T, E, k, scale, flags);
    if (st == MX_ERR_SHAPE) return st;
    if (groups < 1 || groups > MX_ROUTER_MAX_GROUPS || E % groups != 0 || groups_kept < 1 || groups_kept > groups ||
        k > groups_kept * (E / groups) || group_top < 1 || group_top > 2)
        return MX_ERR_SHAPE;
    if (st != MX_OK) return st;
    int32_t padded = 1;
    while (padded < groups) padded *= 2;
    if (groups != padded && E / groups * padded > mx::kRouterSlots) return MX_ERR_UNSUPPORTED;
    if (T == 0) return MX_OK;
    if (!logits || !experts || !weights) return MX_ERR_NULL;
    if (!aligned(logits, flags & MX_ROUTER_LOGITS_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(experts, 4) ||
        !aligned(weights, 4) || !aligned(scores, 4))
        return MX_ERR_ALIGN;
    if ((const void*)scores == logits) return MX_ERR_SHAPE;
    const mx::RouterArgs a{logits, ldl, T, E, bias, groups, groups_kept, group_top, k, scale, flags, experts, weights,
                           scores};
    return from_hip(mx::launch_router(a, (hipStream_t)stream));
}

mx_status mx_router_backward(const void* logits, int64_t ldl, int64_t T, int32_t E, const int32_t* experts,
                             const float* dweights, const float* dscores, int32_t k, float scale, uint32_t flags,
                             void* dlogits, int64_t ldd, void* stream) {
    const mx_status st = check_router(ldl, T, E, k, scale, flags);
    if (st == MX_ERR_SHAPE || k > E || ldd < E) return MX_ERR_SHAPE;
    if (st != MX_OK) return st;
    if (ldd >= kMaxStride) return MX_ERR_UNSUPPORTED;
    if (T == 0) return MX_OK;
    if (!logits || !experts || !dweights || !dlogits) return MX_ERR_NULL;
    const size_t size = flags & MX_ROUTER_LOGITS_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(experts, 4) || !aligned(dweights, 4) ||
        !aligned(dscores, 4))
        return MX_ERR_ALIGN;
    const mx::RouterBackwardArgs a{logits, ldl, T, E, experts, dweights, dscores, k, scale, flags, dlogits, ldd};
    return from_hip(mx::launch_router_backward(a, (hipStream_t)stream));
}

mx_status mx_combine_dweights(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t M, int64_t ldy,
                              const int32_t* slot_of, int64_t T, int32_t k, int64_t N, float* dweights,
                              void* stream) {
    if (M < 0 || N < 0 || T < 0 || k < 1 || ldd < N || ldy < N) return MX_ERR_SHAPE;
    if (ldd % 8 != 0 || ldy % 8 != 0) return MX_ERR_ALIGN;
    if (N % 8 != 0 || T >= kMaxTokens || M >= kMaxRows || T * k >= kMaxRows || ldd >= (int64_t)1 << 30 ||
        ldy >= (int64_t)1 << 30)
        return MX_ERR_UNSUPPORTED;
    if (T == 0) return MX_OK;
    if (!slot_of || !dweights || (N > 0 && (!dout || (M > 0 && !y)))) return MX_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(slot_of, 4) || !aligned(dweights, 4)) return MX_ERR_ALIGN;
    return from_hip(
        mx::launch_combine_dweights(dout, ldd, y, M, ldy, slot_of, T, k, N, dweights, (hipStream_t)stream));
}

mx_status mx_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, int64_t M,
                      int64_t N, float eps, uint32_t flags, void* h, int64_t ldh, uint16_t* y, int64_t ldy,
                      uint8_t* q, uint8_t* s, float* rstd, void* stream) {
    mx_status st = check_norm(M, N, flags);
    if (st == MX_ERR_SHAPE || !(eps >= 0.0f) || !std::isfinite(eps)) return MX_ERR_SHAPE;
    if ((h && !residual) || (q && N % 32 != 0)) return MX_ERR_SHAPE;
    if (st != MX_OK) return st;
    const struct {
        const void* p;
        int64_t ld;
    } rows[] = {{x, ldx}, {residual, ldr}, {h, ldh}, {y, ldy}};
    for (const auto& r : rows)
        if ((st = check_stride(r.p, r.ld, N)) != MX_OK) return st;
    if (M == 0) return MX_OK;
    if (!x || !weight || (residual && !h) || (!q != !s)) return MX_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) || !aligned(y, 16) ||
        !aligned(q, 16) || !aligned(s, 4) || !aligned(rstd, 4))
        return MX_ERR_ALIGN;
    const mx::NormArgs a{x, ldx, residual, ldr, weight, M, N, eps, flags, h, ldh, y, ldy, q, s, rstd};
    return from_hip(mx::launch_rms_norm(a, (hipStream_t)stream));
}

mx_status mx_rms_norm_backward(const uint16_t* dy, int64_t ldy, const uint16_t* dy2, int64_t ldy2, const void* h,
                               int64_t ldh, const void* weight, const float* rstd, const void* dh_in, int64_t ldi,
                               int64_t M, int64_t N, uint32_t flags, void* dh, int64_t ldo, uint16_t* dx, int64_t lddx,
                               void* dweight, int32_t dw_fp32, int32_t accumulate, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    mx_status st = check_norm(M, N, flags);
    if (st == MX_ERR_SHAPE || (dw_fp32 != 0 && dw_fp32 != 1) || (accumulate != 0 && accumulate != 1) ||
        workspace_bytes < 0 || (dx && !(flags & MX_NORM_STREAM_FP32)))
        return MX_ERR_SHAPE;
    if (st != MX_OK) return st;
    if (accumulate && !dw_fp32) return MX_ERR_UNSUPPORTED;
    const struct {
        const void* p;
        int64_t ld;
    } rows[] = {{dy, ldy}, {dy2, ldy2}, {h, ldh}, {dh_in, ldi}, {dh, ldo}, {dx, lddx}};
    for (const auto& r : rows)
        if ((st = check_stride(r.p, r.ld, N)) != MX_OK) return st;
    if (M > 0 && (!dy || !h || !weight || !rstd || !dh)) return MX_ERR_NULL;
    if (M == 0 && (!dweight || accumulate)) return MX_OK;
    if (M > 0 && dweight) {
        const int64_t needed = mx_rms_norm_backward_workspace_bytes(M, N);
        if (workspace_bytes < needed) return MX_ERR_CAPACITY;
        if (needed > 0 && !workspace) return MX_ERR_NULL;
    }
    if (!aligned(dy, 16) || !aligned(dy2, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
        !aligned(dh_in, 16) || !aligned(dh, 16) || !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(workspace, 16))
        return MX_ERR_ALIGN;
    const mx::NormBackwardArgs a{dy, ldy, dy2, ldy2, h, ldh, weight, rstd, dh_in, ldi, M, N, flags, dh, ldo, dx, lddx,
                                 dweight, dw_fp32 != 0, accumulate != 0, (float*)workspace};
    return from_hip(mx::launch_rms_norm_backward(a, (hipStream_t)stream));
}

int64_t mx_rms_norm_backward_workspace_bytes(int64_t M, int64_t N) {
    if (check_norm(M, N, 0) != MX_OK) return -1;
    return mx::norm_backward_needs_parts(M, N) ? 4 * (int64_t)mx::norm_backward_parts(M, N) * N : 0;
}

}  // extern "C"
