// Stand-ins for the launchers of the routed-expert layer (csrc/moe_launch.hpp)
// in the host AddressSanitizer build of csrc/moe_api.cpp: a call that gets past
// validation reaches one of these, which returns an error, so the ABI reports
// MXQ_ERR_HIP and the test that made it fails.  The workspace size is answered
// like the library's: nothing for few slots, something for many.
#include "../../nvfp4_quantization_grouped_amd/csrc/moe_launch.hpp"

namespace mxq {

static hipError_t reached() { return hipErrorNotSupported; }

hipError_t launch_moe_route(const RouteArgs&, int, hipStream_t) { return reached(); }
hipError_t launch_moe_route_bwd(const void*, int, int64_t, int, int, bool, bool, double, const int32_t*, const float*,
                                void*, hipStream_t) {
  return reached();
}
int64_t plan_workspace_bytes(int64_t slots, int local) { return slots <= 1024 ? 0 : int64_t(4) * local; }
hipError_t launch_moe_plan(const int32_t*, int64_t, int, int, int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t) {
  return reached();
}
hipError_t launch_moe_dispatch(const void*, int, int64_t, int64_t, int, const int32_t*, void*, hipStream_t) {
  return reached();
}
hipError_t launch_moe_dispatch_quantized(const void*, int, int64_t, int64_t, int, const int32_t*, int, uint8_t*,
                                         uint8_t*, hipStream_t) {
  return reached();
}
hipError_t launch_moe_combine(const void*, int, int64_t, int64_t, int, const int32_t*, const float*, void*,
                              hipStream_t) {
  return reached();
}
hipError_t launch_moe_combine_bwd(const void*, const void*, int, int64_t, int64_t, int, const int32_t*, const float*,
                                  void*, float*, hipStream_t) {
  return reached();
}
hipError_t launch_swiglu_fwd(const void*, int, int64_t, int64_t, const int32_t*, void*, uint8_t*, uint8_t*,
                             hipStream_t) {
  return reached();
}
hipError_t launch_swiglu_quantized(const void*, int, int64_t, int64_t, const int32_t*, int, uint8_t*, uint8_t*,
                                   hipStream_t) {
  return reached();
}
hipError_t launch_swiglu_bwd(const void*, const void*, const uint8_t*, const uint8_t*, int, int64_t, int64_t,
                             const int32_t*, void*, hipStream_t) {
  return reached();
}

}  // namespace mxq
