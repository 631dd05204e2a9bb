// cache_attention's kernels for mxfp4 pools and f16 queries.
#include "cache_attention.hpp"

namespace mxq {

template <>
hipError_t attention_kernels<DT_F16, FMT_MXFP4>(const AttnArgs* a, int dim, int rows, int64_t problems, AttnShape* shape,
                                     hipStream_t st) {
  return attention_dim<DT_F16, FMT_MXFP4>(a, dim, rows, problems, shape, st);
}

}  // namespace mxq
