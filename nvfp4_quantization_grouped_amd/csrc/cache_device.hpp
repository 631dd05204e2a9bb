// Device-side building blocks of the paged cache's kernels: where a position's
// row lies, and the scale bytes of the three formats.
#pragma once

#include "cache_launch.hpp"
#include "moe_device.hpp"

namespace mxq {

// Scale byte of 2^k as quantize_cache_packed writes it: E8M0 (k + 127) for
// mxfp4 and fp8, E4M3 bits for nvfp4 (k in -9 .. 8, subnormal below -6).
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(int k) {
  if constexpr (FMT == FMT_NVFP4) return k >= -6 ? (uint32_t)(k + 7) << 3 : 1u << (k + 9);
  else return (uint32_t)(k + 127);
}
// Its value; a NaN byte is NaN.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if constexpr (FMT == FMT_NVFP4) return dec_fp8_f2<false>(b, 1.0f).x;
  else return e8m0_to_f32(b);
}

// Cached positions of a sequence: within its row of the table.
__device__ __forceinline__ int cached_positions(int length, int width, int page_size) {
  return min(max(length, 0), width * page_size);
}
// Page of position p of a sequence, or -1.
__device__ __forceinline__ int page_of(const int32_t* __restrict__ row, int width, int page_shift, int64_t pages, int p) {
  const int slot = p >> page_shift;
  if (slot >= width) return -1;
  const int page = row[slot];
  return (uint32_t)page < (uint32_t)pages ? page : -1;
}

inline int log2_of(int v) { return 31 - __builtin_clz((unsigned)v); }

}  // namespace mxq
