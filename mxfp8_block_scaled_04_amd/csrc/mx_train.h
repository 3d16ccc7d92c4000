// What the training-step sources share: the launchers behind
// include/libmxmoe_train.h and the device form of an optimizer plan.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libmxmoe_train.h"

namespace mx {

// Elements of one work item of the optimizer kernels: a workgroup of 4 waves
// takes them as 16 blocks of 256, 4 elements per lane.
constexpr int kAdamwChunk = 4096;

// A tensor as the kernels read it.  first_chunk: the number of chunks before
// it.  The plan is `count` of these, then one int32 per chunk: its tensor.
struct AdamwEntry {
    mx_adamw_tensor t;
    int64_t first_chunk;
};
// type bit added by the plan: every pointer is aligned for 4 elements
constexpr uint32_t kAdamwAligned = 1u << 8;

// Workgroups (and partial sums) of the norm kernel at most.
constexpr int kNormParts = 2048;
struct NormWorkspace {
    double part[kNormParts];
    uint32_t ticket;
    uint32_t pad;
};

struct AdamwArgs {
    const AdamwEntry* entries;
    const int32_t* owner;
    int64_t chunks;
    int64_t* steps;
    const float* lr_device;
    const float* grad_scale;
    double lr, beta1, beta2, eps;
};

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t stream);
hipError_t launch_grad_norm(const AdamwEntry* entries, const int32_t* owner, int64_t chunks, float max_norm,
                            NormWorkspace* ws, float* out, hipStream_t stream);

hipError_t launch_grouped_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* offsets, int32_t G,
                               int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldo, hipStream_t stream);
hipError_t launch_grouped_bf16_dgrad(const uint16_t* dy, int64_t ldy, const uint16_t* w, const int32_t* offsets,
                                     int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* dx, int64_t ldx,
                                     hipStream_t stream);
hipError_t launch_grouped_bf16_wgrad(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                     const int32_t* offsets, int32_t G, int64_t M, int64_t N, int64_t K, void* dw,
                                     bool fp32, bool accumulate, float* workspace, int64_t workspace_bytes,
                                     hipStream_t stream);
// Slices that the rows of each group are cut into for it (1: none).
int32_t wgrad_split(int32_t G, int64_t M, int64_t N, int64_t K);

}  // namespace mx
