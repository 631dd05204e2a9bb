// cache_append: new rows quantized into their places in the pages.
//
// What bounds it is memory: bf16 keys and values [4, 8192, 8, 128] of four
// prompts of different lengths into mxfp4, 93 MB, take 29 us (47 us with one
// row to a thread in the order of the inputs: each row's index took three
// 64-bit divisions, each thread had one load in flight, and its 64 bytes lay
// alone in their page).  The rows of one decoding step take a launch and three
// dependent loads, 3 us.
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

// A workgroup takes a tile of 2^token_shift tokens and as many heads, kPasses rows to a thread: the tokens of a head are
// neighbours in a page, so that a tile's codes and scales lie together there.  Four passes keep four loads of a thread in
// flight (a long prompt 29 us; with 1, 2 and 8 of them 37, 30 and 35).
constexpr int kPasses = 4;

struct AppendDims {
  int tokens, kv_heads, chunk_shift;     // 2^chunk_shift: head_dim / 8
  int width, page_shift, token_shift;
  int token_tiles, head_tiles;
  int64_t pages, tiles;
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
  const int chunk = threadIdx.x & ((1 << d.chunk_shift) - 1), first = threadIdx.x >> d.chunk_shift;
  for (int64_t tile = blockIdx.x; tile < d.tiles; tile += gridDim.x) {
    const int64_t of_heads = tile / d.head_tiles;
    const int b = (int)(of_heads / d.token_tiles);
    const int j0 = (int)(of_heads - (int64_t)b * d.token_tiles) << d.token_shift;
    const int head0 = (int)(tile - of_heads * d.head_tiles) * ((kPasses * kThreads >> d.chunk_shift) >> d.token_shift);
    const int end = counts ? min(counts[b], d.tokens) : d.tokens;
    const int length = cached_positions(lengths[b], d.width, 1 << d.page_shift);
    const int room = (d.width << d.page_shift) - length;     // positions of the table behind them
    const int32_t* row = table + (int64_t)b * d.width;
    Raw8<DT> raw[kPasses];
    int page[kPasses];
    // (a row's lanes go the same way: its block's maximum is taken by all of them)
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int r = first + u * (kThreads >> d.chunk_shift);
      const int j = j0 + (r & ((1 << d.token_shift) - 1)), head = head0 + (r >> d.token_shift);
      page[u] = -1;
      if (j < min(end, room) && head < d.kv_heads) {
        raw[u] = load8<DT, true>(src, (((((int64_t)b * d.tokens + j) * d.kv_heads + head) << d.chunk_shift) + chunk) * 8, 8);
        page[u] = page_of(row, d.width, d.page_shift, d.pages, length + j);
      }
    }
    bool own[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) own[u] = page[u] >= 0 && refs[max(page[u], 0)] == 1;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (!own[u]) continue;
      const int r = first + u * (kThreads >> d.chunk_shift);
      const int j = j0 + (r & ((1 << d.token_shift) - 1)), head = head0 + (r >> d.token_shift);
      float x[8];
      to_f32<DT>(raw[u], x);
      const int e = ceil_rule_exponent<FMT>(group_max_u32<L>(amax_bits(x)));
      const float s = pow2f(e);
      const int64_t at = (((((int64_t)page[u] * d.kv_heads + head) << d.page_shift) +
                           ((length + j) & ((1 << d.page_shift) - 1))) << d.chunk_shift) + chunk;
      if constexpr (FMT == FMT_FP8) *reinterpret_cast<u32x2_t*>(codes + at * 8) = encode_fp8(x, s);
      else *reinterpret_cast<uint32_t*>(codes + at * 4) = encode_fp4(x, s);
      if ((chunk & (L - 1)) == 0) scales[at / L] = (uint8_t)scale_byte<FMT>(e);
    }
  }
}

template <int DT, int FMT>
void launch_blocks(const CacheArgs& c, const TableArgs& t, const void* k, const void* v, const int32_t* counts,
                   const AppendDims& d, hipStream_t st) {
  const dim3 grid((unsigned)min(d.tiles, (int64_t)1 << 20), c.shared ? 1 : 2);
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
  const int chunk_shift = log2_of(c.head_dim / 8), rows = kPasses * kThreads >> chunk_shift;
  int token_shift = 0;
  while ((1 << token_shift) < rows && (1 << token_shift) < tokens) ++token_shift;
  const int heads = rows >> token_shift;
  AppendDims d = {(int)tokens, c.kv_heads, chunk_shift, t.width, log2_of(c.page_size), token_shift,
                  (int)((tokens + (1 << token_shift) - 1) >> token_shift), (c.kv_heads + heads - 1) / heads, c.pages, 0};
  d.tiles = (int64_t)t.sequences * d.token_tiles * d.head_tiles;
  if (dt == DT_F32) launch_formats<DT_F32>(c, t, k, v, counts, d, st);
  else if (dt == DT_BF16) launch_formats<DT_BF16>(c, t, k, v, counts, d, st);
  else launch_formats<DT_F16>(c, t, k, v, counts, d, st);
  return hipGetLastError();
}

}  // namespace mxq
