// cache_attention's kernels for fp8 pools and f16 queries.
#include "cache_attention.hpp"

namespace mxq {

template <>
hipError_t launch_attention_kernels<DT_F16, FMT_FP8>(const AttnArgs& a, int dim, int tiles, int64_t problems, hipStream_t st) {
  return launch_attention_dim<DT_F16, FMT_FP8>(a, dim, tiles, problems, st);
}

}  // namespace mxq
