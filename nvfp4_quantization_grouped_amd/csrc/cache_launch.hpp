// Host-side launchers of the paged cache's kernels (internal; the public ABI is
// include/mxq_pages.h).  Each launcher enqueues on `st` and returns the HIP
// error of the launch.  Arguments are validated by the ABI layer before these
// run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

constexpr int kMaxReserveSequences = 4096;   // what the planning workgroup of cache_reserve holds in LDS

// A cache as the kernels see it.  v pools equal the k pools where the values are the keys.
struct CacheArgs {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int64_t pages;
  int page_size, kv_heads, head_dim, fmt, block;
  bool shared;
};
struct TableArgs {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* refs;
  int sequences, width;
};

hipError_t launch_cache_append(const CacheArgs& c, const TableArgs& t, const void* k, const void* v, int dt,
                               int64_t tokens, const int32_t* counts, hipStream_t st);

struct AttentionArgs {
  const void* q;
  const uint8_t* mask;      // NULL: causal
  const int32_t* counts;    // NULL: all tokens
  void* out;
  float* lse;               // NULL: not wanted
  int tokens, heads;
  bool mask_each;
  float scale;
};
int64_t attention_workspace_bytes(const CacheArgs& c, int64_t sequences, int64_t width, int dt, int64_t tokens,
                                  int64_t heads);
hipError_t launch_cache_attention(const CacheArgs& c, const TableArgs& t, const AttentionArgs& a, int dt,
                                  void* workspace, hipStream_t st);

// parents, keep: NULL for none.
hipError_t launch_cache_fork(const TableArgs& t, int64_t pages, int page_size, const int32_t* parents, int children,
                             const int32_t* keep, bool release, int32_t* table_out, int32_t* lengths_out,
                             int32_t* refs_out, hipStream_t st);
int64_t reserve_workspace_bytes(int64_t sequences, int64_t width, int64_t pages);
hipError_t launch_cache_reserve(const CacheArgs& c, const TableArgs& t, int tokens, const int32_t* tokens_each,
                                int32_t* table_out, int32_t* refs_out, int32_t* short_out, int32_t* workspace,
                                hipStream_t st);
hipError_t launch_cache_accept(const CacheArgs& c, const TableArgs& t, const int32_t* accepted, int most,
                               int32_t* lengths_out, hipStream_t st);
int64_t compact_workspace_bytes(int64_t pages);
hipError_t launch_cache_compact(const CacheArgs& c, const TableArgs& t, int32_t* table_out, int32_t* refs_out,
                                int32_t* workspace, hipStream_t st);

}  // namespace mxq
