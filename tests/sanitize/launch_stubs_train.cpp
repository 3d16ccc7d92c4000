// Host-only stand-ins for the kernel launchers of the training-step calls,
// linked with api_train.cpp into a sanitizer build that runs without a GPU.
// Every stub returns an error: a validation test that reaches one means that
// an entry point let invalid arguments through to a launch.
#include "../../mxfp8_block_scaled_04_amd/csrc/mx_train.h"

namespace mx {

hipError_t launch_adamw(const AdamwArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_grad_norm(const AdamwEntry*, const int32_t*, int64_t, float, NormWorkspace*, float*, hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_grouped_bf16(const uint16_t*, int64_t, const uint16_t*, const int32_t*, int32_t, int64_t, int64_t,
                               int64_t, uint16_t*, int64_t, hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_grouped_bf16_dgrad(const uint16_t*, int64_t, const uint16_t*, const int32_t*, int32_t, int64_t,
                                     int64_t, int64_t, uint16_t*, int64_t, hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_grouped_bf16_wgrad(const uint16_t*, int64_t, const uint16_t*, int64_t, const int32_t*, int32_t,
                                     int64_t, int64_t, int64_t, void*, bool, bool, float*, int64_t, hipStream_t) {
    return hipErrorNotSupported;
}
int32_t wgrad_split(int32_t, int64_t, int64_t, int64_t) { return 2; }

}  // namespace mx
