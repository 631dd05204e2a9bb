// cache_attention's launches: which kernel, and how its work is shared out.
#include "cache_attention.hpp"

namespace mxq {
namespace {

// Steps are shared out among as many workgroups as run at a time.
constexpr int kComputeUnits = 256;
// From so many problems on each has a workgroup of its own: there are enough of them to keep the card busy (8 heads of 512
// sequences of 2048 154 us, 183 shared out; of 256 of 4096 150 and 158; of 128 of 4096 90 and 88).
constexpr int64_t kManyProblems = 2048;
// Below, problems are shared out if they have more steps than a kernel's `few` (14 of 1 us, or 4 of 3 us: what joining
// costs) and this many more for each workgroup's worth of problems.  Of 4 sequences' 8 heads 1024 positions take 16 us, 19
// shared out, 2048 22 and 19; of 32 sequences' 17 and 24, 25 and 29, 3000 35 and 34; of 96 3000 79 and 88; of [4, n, 512] 128
// positions 29 and 26; 16-token trees over 500 positions of 4 sequences 34 and 24, of 32 35 and 41, over 1000 49 and 43.
constexpr int64_t kStepsPerShare = 20;

hipError_t kernels(const AttnArgs* a, int dt, int fmt, int dim, int rows, int64_t problems, AttnShape* shape,
                   hipStream_t st) {
#define FORMATS(DT)                                                                                           \
  if (fmt == FMT_FP8) return attention_kernels<DT, FMT_FP8>(a, dim, rows, problems, shape, st);               \
  if (fmt == FMT_MXFP4) return attention_kernels<DT, FMT_MXFP4>(a, dim, rows, problems, shape, st);           \
  return attention_kernels<DT, FMT_NVFP4>(a, dim, rows, problems, shape, st)
  if (dt == DT_F32) { FORMATS(DT_F32); }
  if (dt == DT_BF16) { FORMATS(DT_BF16); }
  FORMATS(DT_F16);
#undef FORMATS
}

struct Plan {
  int rows;               // of a tile
  int row_tiles;
  int64_t problems;
  int workgroups;         // 0: one for each problem
};
Plan plan_of(const CacheArgs& c, int64_t sequences, int64_t width, int dt, int64_t tokens, int64_t heads) {
  const int64_t rows = tokens * (heads / c.kv_heads);
  Plan p;
  p.rows = attention_rows(c.head_dim, rows);
  p.row_tiles = (int)((rows + p.rows - 1) / p.rows);
  p.problems = sequences * c.kv_heads * p.row_tiles;
  AttnShape shape = {128, 0, 0, 1};
  (void)kernels(nullptr, dt, c.fmt, c.head_dim, p.rows, 0, &shape, nullptr);
  const int64_t steps = (width * c.page_size + shape.step - 1) / shape.step;
  const int workgroups = kComputeUnits * shape.resident;
  const bool split = p.problems < kManyProblems && steps > shape.few + kStepsPerShare * p.problems / workgroups &&
                     p.problems * (steps + shape.start) < (int64_t(1) << 31);
  p.workgroups = split ? workgroups : 0;
  return p;
}

}  // namespace

int64_t attention_workspace_bytes(const CacheArgs& c, int64_t sequences, int64_t width, int dt, int64_t tokens,
                                  int64_t heads) {
  const Plan p = plan_of(c, sequences, width, dt, tokens, heads);
  return (int64_t)p.workgroups * 2 * p.rows * (c.head_dim + 2) * 4;
}

hipError_t launch_cache_attention(const CacheArgs& c, const TableArgs& t, const AttentionArgs& x, int dt,
                                  void* workspace, hipStream_t st) {
  const Plan p = plan_of(c, t.sequences, t.width, dt, x.tokens, x.heads);
  AttnArgs a = {c.k_codes, c.k_scales, c.v_codes, c.v_scales, t.table, t.lengths, x.counts, (const uint8_t*)x.q, x.mask,
                (uint8_t*)x.out, x.lse, (float*)workspace, log2_of(c.block), {}};
  a.d = {t.sequences, x.tokens, x.heads, x.heads / c.kv_heads, c.kv_heads, t.width, log2_of(c.page_size), p.row_tiles,
         p.workgroups, x.mask_each, c.pages, fmaxf((float)(fabs((double)x.scale) * 1.4426950408889634), 0x1p-149f),
         x.scale < 0};
  return kernels(&a, dt, c.fmt, c.head_dim, p.rows, p.problems, nullptr, st);
}

}  // namespace mxq
