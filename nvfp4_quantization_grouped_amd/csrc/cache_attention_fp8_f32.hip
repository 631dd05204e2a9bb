// cache_attention's kernels for fp8 pools and f32 queries.
#include "cache_attention.hpp"

namespace mxq {

template <>
hipError_t attention_kernels<DT_F32, FMT_FP8>(const AttnArgs* a, int dim, int rows, int64_t problems, AttnShape* shape,
                                     hipStream_t st) {
  return attention_dim<DT_F32, FMT_FP8>(a, dim, rows, problems, shape, st);
}

}  // namespace mxq
