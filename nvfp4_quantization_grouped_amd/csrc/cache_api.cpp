// C ABI of the paged cache (declared in include/mxq_pages.h): host-side
// validation, then asynchronous launches on the caller's stream.  No
// allocation, no sync.
#include "../../include/mxq.h"
#include "../../include/mxq_pages.h"
#include "abi_checks.hpp"
#include "cache_launch.hpp"

namespace {

using namespace mxq;

constexpr int64_t kMaxSequences = int64_t(1) << 20;
constexpr int64_t kMaxPositions = int64_t(1) << 30;   // a position and a tile past it fit int32
constexpr int64_t kMaxEntries = int64_t(1) << 30;
constexpr int64_t kMaxRows = int64_t(1) << 36;

bool misaligned16(const void* p) { return ((uintptr_t)p & 15) != 0; }

bool page_size_ok(int64_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

// The sizes of a cache.
int cache_shape(const mxq_cache* c) {
  if (!c) return MXQ_ERR_NULL;
  if (c->pages < 1 || c->pages >= (int64_t(1) << 31) || !page_size_ok(c->page_size) || c->kv_heads < 1 ||
      c->kv_heads > 1024)
    return MXQ_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512) return MXQ_ERR_SHAPE;
  if (c->fmt != MXQ_FMT_FP8 && c->fmt != MXQ_FMT_MXFP4 && c->fmt != MXQ_FMT_NVFP4) return MXQ_ERR_FORMAT;
  if ((c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) || c->block > c->head_dim)
    return MXQ_ERR_BLOCK;
  return MXQ_OK;
}

int table_shape(int64_t sequences, int64_t width, int64_t page_size) {
  if (sequences < 0 || sequences > kMaxSequences || width < 1 || width > kMaxPositions / page_size) return MXQ_ERR_SHAPE;
  return product_below(sequences, width, kMaxEntries) < 0 ? MXQ_ERR_SHAPE : MXQ_OK;
}

// The pools' spans: two or four of them.
struct Pools {
  Span s[4];
  int n;
};
Pools pools_of(const mxq_cache* c) {
  const int64_t rows = c->pages * c->kv_heads * c->page_size;
  const int64_t codes = rows * (c->fmt == MXQ_FMT_FP8 ? c->head_dim : c->head_dim / 2);
  const int64_t scales = rows * (c->head_dim / c->block);
  return {{{c->k_codes, codes}, {c->k_scales, scales}, {c->v_codes, codes}, {c->v_scales, scales}}, c->v_codes ? 4 : 2};
}
int pools_ok(const mxq_cache* c) {
  if (!c->k_codes || !c->k_scales || !c->v_codes != !c->v_scales) return MXQ_ERR_NULL;
  if (misaligned16(c->k_codes) || misaligned16(c->k_scales) || misaligned16(c->v_codes) || misaligned16(c->v_scales))
    return MXQ_ERR_ALIGN;
  return MXQ_OK;
}
// Does a pool that is written overlap another pool, or any of the others?
bool pools_overlap(const mxq_cache* c, const Span* others, int n) {
  const Pools p = pools_of(c);
  for (int i = 0; i < p.n; ++i)
    if (overlaps_any(p.s[i], p.s, i) || overlaps_any(p.s[i], others, n)) return true;
  return false;
}

CacheArgs args_of(const mxq_cache* c) {
  const bool shared = !c->v_codes;
  return {c->k_codes, c->k_scales, shared ? c->k_codes : c->v_codes, shared ? c->k_scales : c->v_scales, c->pages,
          (int)c->page_size, (int)c->kv_heads, (int)c->head_dim, c->fmt, c->block, shared};
}

}  // namespace

extern "C" {

int cache_append(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                 const int32_t* lengths, const int32_t* refs, const void* k, const void* v, int t, int64_t tokens,
                 const int32_t* counts, void* stream) {
  int st = cache_shape(cache);
  if (st == MXQ_OK) st = table_shape(sequences, width, cache->page_size);
  if (st != MXQ_OK) return st;
  if (tokens < 0 || tokens > kMaxSequences) return MXQ_ERR_SHAPE;
  const int64_t rows = product_below(product_below(sequences, tokens, kMaxRows), cache->kv_heads, kMaxRows);
  if (rows < 0) return MXQ_ERR_SHAPE;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (rows == 0) return MXQ_OK;
  st = pools_ok(cache);
  if (st != MXQ_OK) return st;
  if (!table || !lengths || !refs || !k || !v != !cache->v_codes) return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(lengths) || misaligned4(refs) || misaligned4(counts)) return MXQ_ERR_ALIGN;
  const int64_t bytes = rows * cache->head_dim * dtype_bytes(t);
  const Span in[] = {{table, sequences * width * 4}, {lengths, sequences * 4}, {refs, cache->pages * 4}, {k, bytes},
                     {v, bytes}, {counts, sequences * 4}};
  if (pools_overlap(cache, in, 6)) return MXQ_ERR_ALIAS;
  return from_hip(launch_cache_append(args_of(cache), {table, lengths, refs, (int)sequences, (int)width}, k, v, t,
                                      tokens, counts, (hipStream_t)stream));
}

int64_t cache_attention_workspace(const mxq_cache* cache, int64_t sequences, int64_t width, int t, int64_t tokens,
                                  int64_t heads) {
  int st = cache_shape(cache);
  if (st == MXQ_OK) st = table_shape(sequences, width, cache->page_size);
  if (st != MXQ_OK) return st;
  if (tokens < 0 || tokens > 1024 || heads < 1 || heads > (1 << 14) || heads % cache->kv_heads != 0)
    return MXQ_ERR_SHAPE;
  if (product_below(sequences * tokens, heads, (int64_t(1) << 31) - 1) < 0) return MXQ_ERR_SHAPE;
  if (!dtype_ok(t)) return MXQ_ERR_DTYPE;
  if (sequences * tokens == 0) return 0;
  return attention_workspace_bytes(args_of(cache), sequences, width, t, tokens, heads);
}

int cache_attention(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                    const int32_t* lengths, const void* q, int t, int64_t tokens, int64_t heads, const uint8_t* mask,
                    int mask_each, const int32_t* counts, double scale, void* out, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  const int64_t need = cache_attention_workspace(cache, sequences, width, t, tokens, heads);
  if (need < 0) return (int)need;
  if (workspace_bytes < need || !(scale < 0x1p127 && scale > -0x1p127)) return MXQ_ERR_SHAPE;
  const int64_t rows = sequences * tokens * heads;
  if (rows == 0) return MXQ_OK;
  const int st = pools_ok(cache);
  if (st != MXQ_OK) return st;
  if (!table || !lengths || !q || !out || (need > 0 && !workspace)) return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(lengths) || misaligned4(counts) || misaligned4(lse) || misaligned16(q) ||
      misaligned16(out) || misaligned16(workspace))
    return MXQ_ERR_ALIGN;
  const int64_t bytes = rows * cache->head_dim * dtype_bytes(t);
  const Pools p = pools_of(cache);
  Span in[12] = {{table, sequences * width * 4}, {lengths, sequences * 4}, {q, bytes},
                 {mask, tokens * tokens * (mask_each ? sequences : 1)}, {counts, sequences * 4}};
  int n = 5;
  for (int i = 0; i < p.n; ++i) in[n++] = p.s[i];
  const Span outs[] = {{out, bytes}, {lse, rows * 4}, {workspace, need}};
  for (int i = 0; i < 3; ++i)
    if (overlaps_any(outs[i], in, n) || overlaps_any(outs[i], outs, i)) return MXQ_ERR_ALIAS;
  const AttentionArgs a = {q, mask, counts, out, lse, (int)tokens, (int)heads, mask_each != 0, (float)scale};
  return from_hip(launch_cache_attention(args_of(cache), {table, lengths, nullptr, (int)sequences, (int)width}, a, t,
                                         workspace, (hipStream_t)stream));
}

int cache_fork(const int32_t* table, int64_t sequences, int64_t width, const int32_t* lengths, const int32_t* refs,
               int64_t pages, int64_t page_size, const int32_t* parents, int64_t children, const int32_t* keep,
               int release, int32_t* table_out, int32_t* lengths_out, int32_t* refs_out, void* stream) {
  if (!page_size_ok(page_size) || pages < 1 || pages >= (int64_t(1) << 31)) return MXQ_ERR_SHAPE;
  int st = table_shape(sequences, width, page_size);
  if (st == MXQ_OK) st = table_shape(children, width, page_size);
  if (st != MXQ_OK) return st;
  if (!parents && children != sequences && children > 0) return MXQ_ERR_SHAPE;
  if (!refs || !refs_out || (sequences > 0 && (!table || !lengths)) || (children > 0 && (!table_out || !lengths_out)))
    return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(lengths) || misaligned4(refs) || misaligned4(parents) || misaligned4(keep) ||
      misaligned4(table_out) || misaligned4(lengths_out) || misaligned4(refs_out))
    return MXQ_ERR_ALIGN;
  const Span all[] = {{table, sequences * width * 4}, {lengths, sequences * 4}, {refs, pages * 4},
                      {parents, children * 4}, {keep, children * 4}, {table_out, children * width * 4},
                      {lengths_out, children * 4}, {refs_out, pages * 4}};
  for (int i = 5; i < 8; ++i)
    if (overlaps_any(all[i], all, i)) return MXQ_ERR_ALIAS;
  return from_hip(launch_cache_fork({table, lengths, refs, (int)sequences, (int)width}, pages, (int)page_size, parents,
                                    (int)children, keep, release != 0, table_out, lengths_out, refs_out,
                                    (hipStream_t)stream));
}

int64_t cache_reserve_workspace(int64_t sequences, int64_t width, int64_t pages) {
  if (sequences < 0 || sequences > kMaxReserveSequences || width < 1 || width > kMaxPositions / 16 || pages < 1 ||
      pages >= (int64_t(1) << 31) || product_below(sequences, width, kMaxEntries) < 0)
    return MXQ_ERR_SHAPE;
  return reserve_workspace_bytes(sequences, width, pages);
}

int cache_reserve(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                  const int32_t* lengths, const int32_t* refs, int64_t tokens, const int32_t* tokens_each,
                  int32_t* table_out, int32_t* refs_out, int32_t* short_out, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  int st = cache_shape(cache);
  if (st == MXQ_OK) st = table_shape(sequences, width, cache->page_size);
  if (st != MXQ_OK) return st;
  const int64_t need = cache_reserve_workspace(sequences, width, cache->pages);
  if (need < 0 || workspace_bytes < need || tokens > kMaxPositions) return MXQ_ERR_SHAPE;
  st = pools_ok(cache);
  if (st != MXQ_OK) return st;
  if (!refs || !refs_out || (sequences > 0 && (!table || !lengths || !table_out || !short_out)) ||
      !workspace)
    return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(lengths) || misaligned4(refs) || misaligned4(tokens_each) ||
      misaligned4(table_out) || misaligned4(refs_out) || misaligned4(short_out) || misaligned4(workspace))
    return MXQ_ERR_ALIGN;
  const Span all[] = {{table, sequences * width * 4}, {lengths, sequences * 4}, {refs, cache->pages * 4},
                      {tokens_each, sequences * 4}, {table_out, sequences * width * 4}, {refs_out, cache->pages * 4},
                      {short_out, sequences * 4}, {workspace, need}};
  for (int i = 4; i < 8; ++i)
    if (overlaps_any(all[i], all, i)) return MXQ_ERR_ALIAS;
  if (pools_overlap(cache, all, 8)) return MXQ_ERR_ALIAS;
  return from_hip(launch_cache_reserve(args_of(cache), {table, lengths, refs, (int)sequences, (int)width},
                                       (int)(tokens < 0 ? 0 : tokens), tokens_each, table_out, refs_out, short_out,
                                       (int32_t*)workspace, (hipStream_t)stream));
}

int cache_accept(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width,
                 const int32_t* lengths, const int32_t* refs, const int32_t* accepted, int64_t most,
                 int32_t* lengths_out, void* stream) {
  int st = cache_shape(cache);
  if (st == MXQ_OK) st = table_shape(sequences, width, cache->page_size);
  if (st != MXQ_OK) return st;
  if (most < 0 || most > 64) return MXQ_ERR_SHAPE;
  st = pools_ok(cache);
  if (st != MXQ_OK) return st;
  if (sequences == 0) return MXQ_OK;
  if (!table || !lengths || !refs || !lengths_out || (most > 0 && !accepted)) return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(lengths) || misaligned4(refs) || misaligned4(accepted) ||
      misaligned4(lengths_out))
    return MXQ_ERR_ALIGN;
  const Span all[] = {{table, sequences * width * 4}, {lengths, sequences * 4}, {refs, cache->pages * 4},
                      {accepted, sequences * most * 4}, {lengths_out, sequences * 4}};
  if (overlaps_any(all[4], all, 4) || pools_overlap(cache, all, 5)) return MXQ_ERR_ALIAS;
  return from_hip(launch_cache_accept(args_of(cache), {table, lengths, refs, (int)sequences, (int)width}, accepted,
                                      (int)most, lengths_out, (hipStream_t)stream));
}

int64_t cache_compact_workspace(int64_t pages) {
  return pages < 1 || pages >= (int64_t(1) << 31) ? (int64_t)MXQ_ERR_SHAPE : compact_workspace_bytes(pages);
}

int cache_compact(const mxq_cache* cache, const int32_t* table, int64_t sequences, int64_t width, const int32_t* refs,
                  int32_t* table_out, int32_t* refs_out, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = cache_shape(cache);
  if (st == MXQ_OK) st = table_shape(sequences, width, cache->page_size);
  if (st != MXQ_OK) return st;
  const int64_t need = cache_compact_workspace(cache->pages);
  if (workspace_bytes < need) return MXQ_ERR_SHAPE;
  st = pools_ok(cache);
  if (st != MXQ_OK) return st;
  if (!refs || !refs_out || !workspace || (sequences > 0 && (!table || !table_out))) return MXQ_ERR_NULL;
  if (misaligned4(table) || misaligned4(refs) || misaligned4(table_out) || misaligned4(refs_out) ||
      misaligned4(workspace))
    return MXQ_ERR_ALIGN;
  const Span all[] = {{table, sequences * width * 4}, {refs, cache->pages * 4}, {table_out, sequences * width * 4},
                      {refs_out, cache->pages * 4}, {workspace, need}};
  for (int i = 2; i < 5; ++i)
    if (overlaps_any(all[i], all, i)) return MXQ_ERR_ALIAS;
  if (pools_overlap(cache, all, 5)) return MXQ_ERR_ALIAS;
  return from_hip(launch_cache_compact(args_of(cache), {table, nullptr, refs, (int)sequences, (int)width}, table_out,
                                       refs_out, (int32_t*)workspace, (hipStream_t)stream));
}

}  // extern "C"
