// What the sources behind include/libmxmoe_block.h share: their launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libmxmoe_block.h"

namespace mx {

// Experts that a team of 64 lanes holds at most: 64 per lane.
constexpr int kRouterSlots = 4096;

struct RouterArgs {
    const void* logits;
    int64_t ldl;
    int64_t T;
    int32_t E;
    const float* bias;
    int32_t groups, kept, top;
    int32_t k;
    float scale;
    uint32_t flags;
    int32_t* experts;
    float* weights;
    float* scores;
};
hipError_t launch_router(const RouterArgs& a, hipStream_t stream);

struct RouterBackwardArgs {
    const void* logits;
    int64_t ldl;
    int64_t T;
    int32_t E;
    const int32_t* experts;
    const float* dweights;
    const float* dscores;
    int32_t k;
    float scale;
    uint32_t flags;
    void* dlogits;
    int64_t ldd;
};
hipError_t launch_router_backward(const RouterBackwardArgs& a, hipStream_t stream);

hipError_t launch_combine_dweights(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t M, int64_t ldy,
                                   const int32_t* slot_of, int64_t T, int32_t k, int64_t N, float* dweights,
                                   hipStream_t stream);

struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    const void* weight;
    int64_t M, N;
    float eps;
    uint32_t flags;
    void* h;
    int64_t ldh;
    uint16_t* y;
    int64_t ldy;
    uint8_t* q;
    uint8_t* s;
    float* rstd;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

struct NormBackwardArgs {
    const uint16_t* dy;
    int64_t ldy;
    const uint16_t* dy2;
    int64_t ldy2;
    const void* h;
    int64_t ldh;
    const void* weight;
    const float* rstd;
    const void* dh_in;
    int64_t ldi;
    int64_t M, N;
    uint32_t flags;
    void* dh;
    int64_t ldo;
    uint16_t* dx;
    int64_t lddx;
    void* dweight;
    bool dw_fp32, accumulate;
    float* workspace;
};
hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream);
// Rows of partial sums of dweight that its workspace holds, where it is summed from such.
bool norm_backward_needs_parts(int64_t M, int64_t N);
int32_t norm_backward_parts(int64_t M, int64_t N);

}  // namespace mx
