// cache_attention: attention of new tokens over the packed, paged cache.
//
// A wave per row of q: 64 positions at a time, a lane scores one position
// (fp32), the running maximum and sum of the softmax follow, and each lane adds
// its channels of the 64 values.
#include "cache_device.hpp"

namespace mxq {
namespace {

struct AttentionDims {
  int tokens, heads, group, width, page_shift;
  bool mask_each;
  float scale;
};

template <int FMT>
__device__ __forceinline__ float element(const uint8_t* codes, const uint8_t* scales, int64_t row, int dim, int block,
                                         int ch) {
  const float s = scale_value<FMT>(scales[row * (dim / block) + ch / block]);
  if constexpr (FMT == FMT_FP8) return dec_fp8_f2<false>(codes[row * dim + ch], 1.0f).x * s;
  else {
    const uint32_t c = codes[row * (dim / 2) + ch / 2] >> (4 * (ch & 1)) & 15u;
    return bf16_lo(dec_fp4_bf16x2<0>(c, 1.0f)) * s;
  }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(64) k_cache_attention(CacheArgs c, const int32_t* __restrict__ table,
                                                        const int32_t* __restrict__ lengths,
                                                        const uint8_t* __restrict__ q, const uint8_t* __restrict__ mask,
                                                        const int32_t* __restrict__ counts, uint8_t* __restrict__ out,
                                                        float* __restrict__ lse, AttentionDims d) {
  __shared__ float qs[512], ps[64];
  __shared__ int64_t rows[64];
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int head = (int)(row % d.heads), i = (int)(row / d.heads % d.tokens), b = (int)(row / d.heads / d.tokens);
  const int D = c.head_dim, kv = head / d.group;
  const int n = cached_positions(lengths[b], d.width, c.page_size);
  const int count = counts ? min(max(counts[b], 0), d.tokens) : d.tokens;
  for (int ch = lane; ch < D; ch += 64) qs[ch] = elem_value<DT>(load_bits<DT>(q + (row * D + ch) * kElemBytes<DT>));
  __syncthreads();
  float m = -__builtin_inff(), l = 0.0f, acc[8] = {};
  const int end = i < count ? min(n + count, d.width << d.page_shift) : 0;
  for (int p0 = 0; p0 < end; p0 += 64) {
    const int p = p0 + lane, j = p - n;
    bool may = p < end;
    if (may && j >= 0)
      may = mask ? mask[((int64_t)(d.mask_each ? b : 0) * d.tokens + i) * d.tokens + j] != 0 : j <= i;
    const int page = may ? page_of(table + (int64_t)b * d.width, d.width, d.page_shift, c.pages, p) : -1;
    may = page >= 0;
    float s = -__builtin_inff();
    if (may) {
      const int64_t at = (((int64_t)page * c.kv_heads + kv) << d.page_shift) + (p & (c.page_size - 1));
      rows[lane] = at;
      s = 0.0f;
      for (int ch = 0; ch < D; ++ch) s += qs[ch] * element<FMT>(c.k_codes, c.k_scales, at, D, c.block, ch);
      s *= d.scale;
    }
    float top = s;
    for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    const float now = fmaxf(m, top);
    if (__ballot(may) != 0) {
      const float keep = m == -__builtin_inff() ? 0.0f : __expf(m - now);
      const float e = may ? expf(s - now) : 0.0f;
      float sum = e;
      for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
      l = l * keep + sum;
      m = now;
      ps[lane] = may ? e : -1.0f;
      __syncthreads();
      for (int k = 0; k < D / 64; ++k) acc[k] *= keep;
      for (int u = 0; u < 64; ++u) {
        if (ps[u] < 0.0f) continue;
        for (int k = 0; k < D / 64; ++k)
          acc[k] += ps[u] * element<FMT>(c.v_codes, c.v_scales, rows[u], D, c.block, lane + 64 * k);
      }
    }
    __syncthreads();
  }
  for (int k = 0; k < D / 64; ++k)
    store_bits<DT>(out + (row * D + lane + 64 * k) * kElemBytes<DT>, elem_bits<DT>(l == 0.0f ? 0.0f : acc[k] / l));
  if (lse && lane == 0) lse[row] = l == 0.0f ? -__builtin_inff() : m + logf(l);
}

}  // namespace

int64_t attention_workspace_bytes(const CacheArgs&, int64_t, int64_t, int, int64_t, int64_t) { return 0; }

hipError_t launch_cache_attention(const CacheArgs& c, const TableArgs& t, const AttentionArgs& a, int dt, void*,
                                  hipStream_t st) {
  const AttentionDims d = {a.tokens, a.heads, a.heads / c.kv_heads, t.width, log2_of(c.page_size), a.mask_each,
                           a.scale};
  const int64_t rows = (int64_t)t.sequences * a.tokens * a.heads;
#define CALL(DT, FMT)                                                                                              \
  k_cache_attention<DT, FMT><<<(unsigned)rows, 64, 0, st>>>(c, t.table, t.lengths, (const uint8_t*)a.q, a.mask,    \
                                                            a.counts, (uint8_t*)a.out, a.lse, d)
#define FORMATS(DT)                                   \
  if (c.fmt == FMT_FP8) CALL(DT, FMT_FP8);            \
  else if (c.fmt == FMT_MXFP4) CALL(DT, FMT_MXFP4);   \
  else CALL(DT, FMT_NVFP4)
  if (dt == DT_F32) { FORMATS(DT_F32); }
  else if (dt == DT_BF16) { FORMATS(DT_BF16); }
  else { FORMATS(DT_F16); }
#undef FORMATS
#undef CALL
  return hipGetLastError();
}

}  // namespace mxq
