// Host-only stand-ins for the kernel launchers of the router's and the norm's
// calls, linked with api_block.cpp into a sanitizer build that runs without a
// GPU.  Every stub returns an error: a validation test that reaches one means
// that an entry point let invalid arguments through to a launch.
#include "../../mxfp8_block_scaled_04_amd/csrc/mx_block.h"

namespace mx {

hipError_t launch_router(const RouterArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_router_backward(const RouterBackwardArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_combine_dweights(const uint16_t*, int64_t, const uint16_t*, int64_t, int64_t, const int32_t*, int64_t,
                                   int32_t, int64_t, float*, hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_rms_norm(const NormArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_rms_norm_backward(const NormBackwardArgs&, hipStream_t) { return hipErrorNotSupported; }
bool norm_backward_needs_parts(int64_t M, int64_t) { return M > 256; }
int32_t norm_backward_parts(int64_t M, int64_t) { return M < 4 ? (int32_t)M : 4; }

}  // namespace mx
