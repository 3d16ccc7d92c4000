// C-ABI entry points of the training step: argument validation, then the
// launchers.  See include/libmxmoe_train.h for the contract of each call.
#include "../../include/libmxmoe_train.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "mx_train.h"

namespace {

bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }

mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

constexpr int32_t kMaxGroups = 4096;
// A tile's operand and output addresses are 32-bit offsets from a 64-bit
// base: 256 rows of a stride below 2^22 elements stay below 2^32 bytes.
constexpr int64_t kMaxDim = (int64_t)1 << 22;

// What the three products share: sizes, row strides of the two row-major
// [M] operands or results (a: width wa, b: width wb) and the group count.
mx_status check_product(int32_t G, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t wa, int64_t ldb, int64_t wb) {
    if (M < 0 || N < 0 || K < 0 || N % 8 != 0 || K % 8 != 0 || lda < wa || ldb < wb) return MX_ERR_SHAPE;
    if (G < 1 || G > kMaxGroups) return MX_ERR_SHAPE;
    if (lda % 8 != 0 || ldb % 8 != 0) return MX_ERR_ALIGN;
    if (N >= kMaxDim || K >= kMaxDim || lda >= kMaxDim || ldb >= kMaxDim || M >= ((int64_t)1 << 31) ||
        N * K >= ((int64_t)1 << 31))
        return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

int64_t chunks_of(int64_t n) { return (n + mx::kAdamwChunk - 1) / mx::kAdamwChunk; }

// The chunks of a list, or -1.
int64_t count_chunks(const mx_adamw_tensor* tensors, int32_t count) {
    if (count < 0 || (count > 0 && !tensors)) return -1;
    int64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (tensors[i].n < 0 || tensors[i].n > INT64_MAX / 2) return -1;
        chunks += chunks_of(tensors[i].n);
        if (chunks > INT32_MAX) return -1;
    }
    return chunks;
}

}  // namespace

extern "C" {

mx_status mx_grouped_gemm_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* group_offsets,
                               int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldo, void* stream) {
    const mx_status s = check_product(G, M, N, K, ldx, K, ldo, N);
    if (s != MX_OK) return s;
    if (M == 0 || N == 0) return MX_OK;
    if (!group_offsets || !out || (K > 0 && (!x || !w))) return MX_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(group_offsets, 4)) return MX_ERR_ALIGN;
    return from_hip(mx::launch_grouped_bf16(x, ldx, w, group_offsets, G, M, N, K, out, ldo, (hipStream_t)stream));
}

mx_status mx_grouped_gemm_bf16_dgrad(const uint16_t* dy, int64_t ldy, const uint16_t* w, const int32_t* group_offsets,
                                     int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* dx, int64_t ldx,
                                     void* stream) {
    const mx_status s = check_product(G, M, N, K, ldy, N, ldx, K);
    if (s != MX_OK) return s;
    if (M == 0 || K == 0) return MX_OK;
    if (!group_offsets || !dx || (N > 0 && (!dy || !w))) return MX_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16) || !aligned(group_offsets, 4)) return MX_ERR_ALIGN;
    return from_hip(
        mx::launch_grouped_bf16_dgrad(dy, ldy, w, group_offsets, G, M, N, K, dx, ldx, (hipStream_t)stream));
}

mx_status mx_grouped_gemm_bf16_wgrad(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                     const int32_t* group_offsets, int32_t G, int64_t M, int64_t N, int64_t K,
                                     void* dw, int32_t dw_fp32, int32_t accumulate, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
    const mx_status s = check_product(G, M, N, K, ldy, N, ldx, K);
    if (s != MX_OK) return s;
    if ((dw_fp32 != 0 && dw_fp32 != 1) || (accumulate != 0 && accumulate != 1) || workspace_bytes < 0)
        return MX_ERR_SHAPE;
    if (accumulate && !dw_fp32) return MX_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return MX_OK;
    if (!group_offsets || !dw || (M > 0 && (!dy || !x))) return MX_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(group_offsets, 4) ||
        !aligned(workspace, 16))
        return MX_ERR_ALIGN;
    return from_hip(mx::launch_grouped_bf16_wgrad(dy, ldy, x, ldx, group_offsets, G, M, N, K, dw, dw_fp32 != 0,
                                                  accumulate != 0, (float*)workspace, workspace_bytes,
                                                  (hipStream_t)stream));
}

int64_t mx_grouped_gemm_bf16_wgrad_workspace_bytes(int32_t G, int64_t M, int64_t N, int64_t K) {
    if (check_product(G, M, N, K, N, N, K, K) != MX_OK) return -1;
    const int32_t split = mx::wgrad_split(G, M, N, K);
    return split > 1 ? 4 * (int64_t)split * G * N * K : 0;
}

int64_t mx_adamw_plan_bytes(const mx_adamw_tensor* tensors, int32_t count) {
    const int64_t chunks = count_chunks(tensors, count);
    if (chunks < 0) return -1;
    return (int64_t)sizeof(mx::AdamwEntry) * count + 4 * chunks;
}

mx_status mx_adamw_plan(const mx_adamw_tensor* tensors, int32_t count, void* plan, int64_t* chunks) {
    if (count < 0) return MX_ERR_SHAPE;
    if (!chunks || (count > 0 && (!tensors || !plan))) return MX_ERR_NULL;
    for (int32_t i = 0; i < count; ++i) {
        const mx_adamw_tensor& t = tensors[i];
        const bool wb = t.types & MX_ADAMW_W_BF16, gb = t.types & MX_ADAMW_G_BF16, s8 = t.types & MX_ADAMW_STATE_8BIT;
        if (t.n < 0 || t.n > INT64_MAX / 2) return MX_ERR_SHAPE;
        if ((t.types & ~(uint32_t)(MX_ADAMW_W_BF16 | MX_ADAMW_G_BF16 | MX_ADAMW_STATE_8BIT | MX_ADAMW_UNBIASED)) != 0)
            return MX_ERR_SHAPE;
        if ((t.master && !wb) || !(t.weight_decay >= 0.0f) || !std::isfinite(t.weight_decay)) return MX_ERR_SHAPE;
        if (!s8 && (t.m_scale || t.v_scale || (t.types & MX_ADAMW_UNBIASED))) return MX_ERR_SHAPE;
        if (t.n == 0) continue;
        if (!t.w || !t.g || !t.m || !t.v || (s8 && (!t.m_scale || !t.v_scale))) return MX_ERR_NULL;
        const size_t state = s8 ? 1 : 4;
        if (!aligned(t.w, wb ? 2 : 4) || !aligned(t.master, 4) || !aligned(t.g, gb ? 2 : 4) || !aligned(t.m, state) ||
            !aligned(t.v, state) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
            return MX_ERR_ALIGN;
    }
    const int64_t total = count_chunks(tensors, count);
    if (total < 0) return MX_ERR_UNSUPPORTED;
    char* const entries = (char*)plan;
    char* const owner = entries + sizeof(mx::AdamwEntry) * (size_t)count;
    int64_t at = 0;
    for (int32_t i = 0; i < count; ++i) {
        mx::AdamwEntry e;
        std::memset(&e, 0, sizeof e);
        e.t = tensors[i];
        e.first_chunk = at;
        const bool wb = e.t.types & MX_ADAMW_W_BF16, gb = e.t.types & MX_ADAMW_G_BF16,
                   s8 = e.t.types & MX_ADAMW_STATE_8BIT;
        const size_t state = s8 ? 4 : 16;
        if (aligned(e.t.w, wb ? 8 : 16) && aligned(e.t.master, 16) && aligned(e.t.g, gb ? 8 : 16) &&
            aligned(e.t.m, state) && aligned(e.t.v, state))
            e.t.types |= mx::kAdamwAligned;
        std::memcpy(entries + sizeof e * (size_t)i, &e, sizeof e);
        for (int64_t c = chunks_of(e.t.n); c > 0; --c, ++at) std::memcpy(owner + 4 * at, &i, 4);
    }
    *chunks = total;
    return MX_OK;
}

int64_t mx_grad_norm_workspace_bytes(void) { return (int64_t)sizeof(mx::NormWorkspace); }

mx_status mx_grad_norm(const void* plan, int32_t count, int64_t chunks, float max_norm, void* workspace, float* out,
                       void* stream) {
    if (count < 0 || chunks < 0 || chunks > INT32_MAX || !(max_norm > 0.0f)) return MX_ERR_SHAPE;
    if (!workspace || !out || (chunks > 0 && !plan)) return MX_ERR_NULL;
    if (!aligned(plan, 16) || !aligned(workspace, 8) || !aligned(out, 4)) return MX_ERR_ALIGN;
    const mx::AdamwEntry* const entries = (const mx::AdamwEntry*)plan;
    return from_hip(mx::launch_grad_norm(entries, (const int32_t*)(entries + count), chunks, max_norm,
                                         (mx::NormWorkspace*)workspace, out, (hipStream_t)stream));
}

mx_status mx_adamw(const void* plan, int32_t count, int64_t chunks, int64_t* steps, double lr, const float* lr_device,
                   double beta1, double beta2, double eps, const float* grad_scale, void* stream) {
    if (count < 0 || chunks < 0 || chunks > INT32_MAX) return MX_ERR_SHAPE;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        !std::isfinite(lr))
        return MX_ERR_SHAPE;
    if (!steps || (chunks > 0 && !plan)) return MX_ERR_NULL;
    if (!aligned(plan, 16) || !aligned(steps, 8) || !aligned(lr_device, 4) || !aligned(grad_scale, 4))
        return MX_ERR_ALIGN;
    mx::AdamwArgs a;
    a.entries = (const mx::AdamwEntry*)plan;
    a.owner = (const int32_t*)(a.entries + count);
    a.chunks = chunks;
    a.steps = steps;
    a.lr_device = lr_device;
    a.grad_scale = grad_scale;
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    return from_hip(mx::launch_adamw(a, (hipStream_t)stream));
}

}  // extern "C"
