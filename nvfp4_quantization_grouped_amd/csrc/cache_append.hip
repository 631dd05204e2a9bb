// cache_append: new rows quantized into their places in the pages.
//
// One pass: a row's channels are read once (non-temporal, nobody reads them
// again), 8 to a lane; the lanes of a block find its largest magnitude by DPP,
// and codes and scale bytes go to the row's place in the page.  The rule is
// quantize_cache_packed's (power-of-two ceiling, nearest-even), with the same
// device functions, so the bytes are the same.
#include "cache_device.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 256;

struct AppendDims {
  int tokens, kv_heads, chunks;     // chunks: head_dim / 8
  int width, page_shift;
  int64_t pages, items;             // items: sequences * tokens * kv_heads * chunks
};

// L lanes of 8 channels share a scale.
template <int DT, int FMT, int L>
__global__ void __launch_bounds__(kThreads) k_cache_append(CacheArgs c, const int32_t* __restrict__ table,
                                                           const int32_t* __restrict__ lengths,
                                                           const int32_t* __restrict__ refs,
                                                           const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                                                           const int32_t* __restrict__ counts, AppendDims d) {
  const uint8_t* src = blockIdx.y ? v : k;
  uint8_t* codes = blockIdx.y ? c.v_codes : c.k_codes;
  uint8_t* scales = blockIdx.y ? c.v_scales : c.k_scales;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < d.items; i += (int64_t)gridDim.x * kThreads) {
    // the lanes of a block take every step together: items and a workgroup's first one are multiples of 8
    const int64_t row = i / d.chunks;
    const int chunk = (int)(i - row * d.chunks);
    const int64_t token = row / d.kv_heads;
    const int head = (int)(row - token * d.kv_heads);
    const int b = (int)(token / d.tokens), j = (int)(token - (int64_t)b * d.tokens);
    if (counts && j >= counts[b]) continue;
    const int64_t p = (int64_t)cached_positions(lengths[b], d.width, 1 << d.page_shift) + j;
    if (p >= (int64_t)d.width << d.page_shift) continue;
    const int page = page_of(table + (int64_t)b * d.width, d.width, d.page_shift, d.pages, (int)p);
    if (page < 0 || refs[page] != 1) continue;
    float x[8];
    to_f32<DT>(load8<DT, true>(src, i * 8, 8), x);
    const int e = ceil_rule_exponent<FMT>(group_max_u32<L>(amax_bits(x)));
    const float s = pow2f(e);
    const int64_t at = ((((int64_t)page * d.kv_heads + head) << d.page_shift) + ((int)p & ((1 << d.page_shift) - 1))) *
                           d.chunks + chunk;
    if constexpr (FMT == FMT_FP8) *reinterpret_cast<u32x2_t*>(codes + at * 8) = encode_fp8(x, s);
    else *reinterpret_cast<uint32_t*>(codes + at * 4) = encode_fp4(x, s);
    if ((chunk & (L - 1)) == 0) scales[at / L] = (uint8_t)scale_byte<FMT>(e);
  }
}

template <int DT, int FMT>
void launch_blocks(const CacheArgs& c, const TableArgs& t, const void* k, const void* v, const int32_t* counts,
                   const AppendDims& d, hipStream_t st) {
  const dim3 grid((unsigned)min((d.items + kThreads - 1) / kThreads, (int64_t)1 << 20), c.shared ? 1 : 2);
#define CALL(L)                                                                                                    \
  k_cache_append<DT, FMT, L><<<grid, kThreads, 0, st>>>(c, t.table, t.lengths, t.refs, (const uint8_t*)k,          \
                                                        (const uint8_t*)v, counts, d)
  if (c.block == 16) CALL(2);
  else if (c.block == 32) CALL(4);
  else if (c.block == 64) CALL(8);
  else CALL(16);
#undef CALL
}

template <int DT>
void launch_formats(const CacheArgs& c, const TableArgs& t, const void* k, const void* v, const int32_t* counts,
                    const AppendDims& d, hipStream_t st) {
  if (c.fmt == FMT_FP8) launch_blocks<DT, FMT_FP8>(c, t, k, v, counts, d, st);
  else if (c.fmt == FMT_MXFP4) launch_blocks<DT, FMT_MXFP4>(c, t, k, v, counts, d, st);
  else launch_blocks<DT, FMT_NVFP4>(c, t, k, v, counts, d, st);
}

}  // namespace

hipError_t launch_cache_append(const CacheArgs& c, const TableArgs& t, const void* k, const void* v, int dt,
                               int64_t tokens, const int32_t* counts, hipStream_t st) {
  AppendDims d = {(int)tokens, c.kv_heads, c.head_dim / 8, t.width, log2_of(c.page_size), c.pages, 0};
  d.items = t.sequences * tokens * c.kv_heads * d.chunks;
  if (dt == DT_F32) launch_formats<DT_F32>(c, t, k, v, counts, d, st);
  else if (dt == DT_BF16) launch_formats<DT_BF16>(c, t, k, v, counts, d, st);
  else launch_formats<DT_F16>(c, t, k, v, counts, d, st);
  return hipGetLastError();
}

}  // namespace mxq
