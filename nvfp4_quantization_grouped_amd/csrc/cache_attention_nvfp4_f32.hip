// cache_attention's kernels for nvfp4 pools and f32 queries.
#include "cache_attention.hpp"

namespace mxq {

template <>
hipError_t launch_attention_kernels<DT_F32, FMT_NVFP4>(const AttnArgs& a, int dim, int tiles, int64_t problems, hipStream_t st) {
  return launch_attention_dim<DT_F32, FMT_NVFP4>(a, dim, tiles, problems, st);
}

}  // namespace mxq
