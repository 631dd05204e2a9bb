// Stand-ins for the launchers of the paged cache (csrc/cache_launch.hpp) in the
// host AddressSanitizer build of csrc/cache_api.cpp: a call that gets past
// validation reaches one of these, which returns an error, so the ABI reports
// MXQ_ERR_HIP and the test that made it fails.  Workspace sizes are of the
// library's kind: something for every call.
#include "../../nvfp4_quantization_grouped_amd/csrc/cache_launch.hpp"

namespace mxq {

static hipError_t reached() { return hipErrorNotSupported; }

hipError_t launch_cache_append(const CacheArgs&, const TableArgs&, const void*, const void*, int, int64_t,
                               const int32_t*, hipStream_t) {
  return reached();
}
int64_t attention_workspace_bytes(const CacheArgs&, int64_t, int64_t, int, int64_t, int64_t) { return 1024; }
hipError_t launch_cache_attention(const CacheArgs&, const TableArgs&, const AttentionArgs&, int, void*, hipStream_t) {
  return reached();
}
hipError_t launch_cache_fork(const TableArgs&, int64_t, int, const int32_t*, int, const int32_t*, bool, int32_t*,
                             int32_t*, int32_t*, hipStream_t) {
  return reached();
}
int64_t reserve_workspace_bytes(int64_t sequences, int64_t, int64_t) { return 4 * (1 + 3 * sequences); }
hipError_t launch_cache_reserve(const CacheArgs&, const TableArgs&, int, const int32_t*, int32_t*, int32_t*, int32_t*,
                                int32_t*, hipStream_t) {
  return reached();
}
hipError_t launch_cache_accept(const CacheArgs&, const TableArgs&, const int32_t*, int, int32_t*, hipStream_t) {
  return reached();
}
int64_t compact_workspace_bytes(int64_t pages) { return 4 * (4 + 2 * pages); }
hipError_t launch_cache_compact(const CacheArgs&, const TableArgs&, int32_t*, int32_t*, int32_t*, hipStream_t) {
  return reached();
}

}  // namespace mxq
