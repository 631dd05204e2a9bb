// The pages of the packed cache between two steps of a serving loop: forking
// and freeing (table rows and counts), reserving (free pages, and copies of
// shared ones that are about to be written), moving accepted rows together,
// and compacting the pool.
//
// The tables are small, so what these calls cost is launches and dependent
// loads, not bytes: each is one or two launches.  Whatever depends on an order
// (which sequence gets which free page) is decided by one workgroup with prefix
// sums; counts are integer atomics, whose sum does not depend on their order.
// Measured: fork 3 us, the plan of a reserve 9 to 11 (four loads in a row, three
// more round trips where pages are shared, then the scans over the sequences and
// the pages) and its copies 4 to 9, accept 3.6, the plan of a compaction 6; its
// copies 13 us for 55 MB, 4.2 TB/s.
#include "cache_device.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPagesPerThread = 16;

__device__ __forceinline__ bool valid_page(int page, int64_t pages) { return (uint32_t)page < (uint32_t)pages; }

// Sum over the lanes below this one; the wave's total in `total`.
__device__ __forceinline__ int wave_scan(int v, int& total) {
  int x = v;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int y = __shfl_up(x, s);
    if ((int)(threadIdx.x & 63) >= s) x += y;
  }
  total = __shfl(x, 63);
  return x - v;
}
// Sum over the threads below this one, of the planning workgroup.  sums: LDS, kPlanWaves entries.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  int wave_total;
  int below = wave_scan(v, wave_total);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = wave_total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < (int)(threadIdx.x >> 6)) below += sums[w];
    total += sums[w];
  }
  return below;
}

// Which of the thread's kPagesPerThread pages from `first` on are used (refs > 0), one bit each; `exist`: which exist.
__device__ __forceinline__ uint32_t used_pages(const int32_t* __restrict__ refs, int64_t first, int64_t pages,
                                               uint32_t& exist) {
  uint32_t used = 0;
  exist = 0;
  if (first + kPagesPerThread <= pages) {
    exist = (1u << kPagesPerThread) - 1;
#pragma unroll
    for (int i = 0; i < kPagesPerThread / 4; ++i) {
      const u32x4_t r = *reinterpret_cast<const u32x4_any*>(refs + first + 4 * i);
      used |= (uint32_t)((int)r.x > 0) << (4 * i) | (uint32_t)((int)r.y > 0) << (4 * i + 1) |
              (uint32_t)((int)r.z > 0) << (4 * i + 2) | (uint32_t)((int)r.w > 0) << (4 * i + 3);
    }
  } else {
    for (int i = 0; i < kPagesPerThread && first + i < pages; ++i) {
      exist |= 1u << i;
      used |= (uint32_t)(refs[first + i] > 0) << i;
    }
  }
  return used;
}

// ------------------------------------------------------------- fork and free
struct ForkDims {
  int64_t pages;
  int sequences, children, width, page_shift;
  bool release;
};

struct ForkArgs {
  const int32_t *table, *lengths, *refs, *parents, *keep;
  int32_t *table_out, *lengths_out, *refs_out;
};
// Entry `slot` of child's row, and the child's length.
__device__ __forceinline__ int forked(const ForkArgs& a, const ForkDims& d, int child, int slot, int& length) {
  const int parent = a.parents ? a.parents[child] : child;
  const bool known = (uint32_t)parent < (uint32_t)d.sequences;
  int page = known ? a.table[(int64_t)parent * d.width + slot] : -1;
  length = known ? a.lengths[parent] : 0;
  if (a.keep) {
    length = min(length, max(a.keep[child], 0));
    const int64_t last = ((int64_t)max(length, 0) + (1 << d.page_shift) - 1) >> d.page_shift;
    if (slot >= last) page = -1;
  }
  return valid_page(page, d.pages) ? page : -1;
}

// Small tables in one launch: the first workgroups count, each the entries that name one of its pages (it looks at all of
// them), the others write the rows.
constexpr int kOwnPages = 1024;
__global__ void __launch_bounds__(kPlanThreads) k_cache_fork_once(ForkArgs a, ForkDims d, int counting) {
  const int entries = d.children * d.width, tid = threadIdx.x;
  int length;
  if ((int)blockIdx.x >= counting) {
    const int step = ((int)gridDim.x - counting) * kPlanThreads;
    for (int i = ((int)blockIdx.x - counting) * kPlanThreads + tid; i < entries; i += step) {
      const int child = i / d.width, slot = i - child * d.width;
      a.table_out[i] = forked(a, d, child, slot, length);
      if (slot == 0) a.lengths_out[child] = length;
    }
    return;
  }
  __shared__ int counts[kOwnPages];
  const int64_t first = (int64_t)blockIdx.x * kOwnPages;
  for (int i = tid; i < kOwnPages; i += kPlanThreads) counts[i] = first + i < d.pages ? a.refs[first + i] : 0;
  __syncthreads();
  // (a page is below `pages`, and -1 lies below every first one)
  auto count = [&](int page, int by) {
    const int64_t at = page - first;
    if (at >= 0 && at < kOwnPages) atomicAdd(counts + at, by);
  };
#pragma unroll 4
  for (int i = tid; i < entries; i += kPlanThreads) {
    const int child = i / d.width;
    count(forked(a, d, child, i - child * d.width, length), 1);
  }
  const int gone = d.release ? d.sequences * d.width : 0;
#pragma unroll 4
  for (int i = tid; i < gone; i += kPlanThreads) {
    const int page = a.table[i];
    if (valid_page(page, d.pages)) count(page, -1);
  }
  __syncthreads();
  for (int i = tid; i < kOwnPages; i += kPlanThreads)
    if (first + i < d.pages) a.refs_out[first + i] = counts[i];
}

// Large ones in two: rows and the old counts, then the entries are counted.
__global__ void __launch_bounds__(kThreads) k_cache_fork(ForkArgs a, ForkDims d) {
  const int64_t entries = (int64_t)d.children * d.width;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < d.pages; i += step) a.refs_out[i] = a.refs[i];
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < entries; i += step) {
    const int child = (int)(i / d.width), slot = (int)(i - (int64_t)child * d.width);
    int length;
    a.table_out[i] = forked(a, d, child, slot, length);
    if (slot == 0) a.lengths_out[child] = length;
  }
}

__global__ void __launch_bounds__(kThreads) k_cache_fork_count(ForkArgs a, ForkDims d) {
  const int64_t added = (int64_t)d.children * d.width, gone = d.release ? (int64_t)d.sequences * d.width : 0;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < added + gone; i += (int64_t)gridDim.x * kThreads) {
    const int page = i < added ? a.table_out[i] : a.table[i - added];
    if (valid_page(page, d.pages)) atomicAdd(a.refs_out + page, i < added ? 1 : -1);
  }
}

// ------------------------------------------------------------------- reserve
struct ReserveDims {
  int64_t pages;
  int sequences, width, page_shift, tokens;
};
// int32 arrays of the workspace: [0] pages granted, then per sequence its first rank among the wanted pages; per page (of
// those that shared entries ask for) how many ask, and the last that does; then the free pages in rising order.
struct ReserveSpace {
  int32_t *granted, *rank, *asks, *last, *free;
};
__host__ __device__ inline ReserveSpace reserve_space(int32_t* w, int sequences, int64_t pages) {
  return {w, w + 1, w + 1 + sequences, w + 1 + sequences + pages, w + 1 + sequences + 2 * pages};
}

// What a sequence asks for.
struct Need {
  int length, slot, end;         // slots slot .. end - 1 must have pages of the sequence's own
  int beyond;                    // pages for which the table has no room
};
__device__ __forceinline__ Need need_of(int length, int tokens, const ReserveDims& d) {
  Need n;
  n.length = cached_positions(length, d.width, 1 << d.page_shift);
  n.slot = n.length >> d.page_shift;
  const int64_t end = ((int64_t)n.length + max(tokens, 0) + (1 << d.page_shift) - 1) >> d.page_shift;
  n.beyond = (int)max(end - d.width, (int64_t)0);
  n.end = tokens > 0 ? (int)min(end, (int64_t)d.width) : 0;
  return n;
}

// Memory that the planning workgroup's waves share among themselves, in order across its barriers.  (Fences for the whole
// device write back the L2 as well: a fork and a reserve of 64 beams, alone, 62 us with them and 51 without.)
__device__ __forceinline__ int shared_load(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void shared_store(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// Workgroup 0 plans; the others copy the table and the counts, which the second launch changes.
//
// An entry that asks for a page which others name too (refs > 1) gets another one, unless it is the last to ask and all
// that name the page ask.  So each page needs two numbers, how many entries ask and which is the last: a count and a
// maximum, whose order does not matter, where comparing the entries would take the square of their number (a token each for
// 1024 beams of four 27 us with both launches, 41 by comparing; 4096 of them 89 and 295).
__global__ void __launch_bounds__(kPlanThreads) k_cache_reserve_plan(const int32_t* __restrict__ table,
                                                                     const int32_t* __restrict__ lengths,
                                                                     const int32_t* __restrict__ refs,
                                                                     const int32_t* __restrict__ tokens_each,
                                                                     int32_t* __restrict__ table_out,
                                                                     int32_t* __restrict__ refs_out, int32_t* work,
                                                                     ReserveDims d) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int64_t entries = (int64_t)d.sequences * d.width, step = (int64_t)(gridDim.x - 1) * kPlanThreads;
    const int64_t first = (int64_t)(blockIdx.x - 1) * kPlanThreads + tid;
    for (int64_t i = first; i < d.pages; i += step) refs_out[i] = refs[i];
    for (int64_t i = first; i < entries; i += step) {
      const int page = table[i];
      table_out[i] = valid_page(page, d.pages) ? page : -1;
    }
    return;
  }
  const ReserveSpace w = reserve_space(work, d.sequences, d.pages);
  __shared__ int wants[kMaxReserveSequences];     // free pages a sequence wants, then its first rank among all
  __shared__ int sums[kPlanWaves];
  // as many lanes to a sequence, side by side, as let all sequences go at once
  const int shift = min(max(31 - __builtin_clz(kPlanThreads / max(d.sequences, 1) | 1), 0), 6), lanes = 1 << shift;
  const int lane = tid & (lanes - 1);
  const uint64_t group = (lanes == 64 ? ~0ull : (1ull << lanes) - 1) << (tid & 63 & ~(lanes - 1));
  const uint64_t below_me = (1ull << (tid & 63)) - 1;
  // f(entry of the table, whether it is asked for, its page or -1, refs of the page or 0), the lanes of a sequence at its
  // entries in turn; begin(sequence) and end(sequence) around them.  A lane's loads go out kAtOnce entries at a time.
  constexpr int kAtOnce = 4;
  auto walk = [&](auto begin, auto f, auto end) {
    for (int b = tid >> shift; b < d.sequences; b += kPlanThreads >> shift) {
      const Need n = need_of(lengths[b], tokens_each ? tokens_each[b] : d.tokens, d);
      begin(b);
      for (int s0 = n.slot; s0 < n.end; s0 += lanes * kAtOnce) {
        int page[kAtOnce], held[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int s = s0 + u * lanes + lane;
          page[u] = s < n.end ? table[(int64_t)b * d.width + s] : -1;
          page[u] = valid_page(page[u], d.pages) ? page[u] : -1;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) held[u] = page[u] >= 0 ? refs[page[u]] : 0;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int s = s0 + u * lanes + lane;
          f(b * d.width + s, s < n.end, page[u], held[u]);
        }
      }
      end(b);
    }
  };
  bool found_shared = false;
  int missing = 0;
  walk([&](int) { missing = 0; },
       [&](int, bool in, int page, int held) {
         missing += __popcll(__ballot(in && page < 0) & group);
         if (held > 1) {
           found_shared = true;
           shared_store(w.asks + page, 0);
           shared_store(w.last + page, -1);
         }
       },
       [&](int b) {
         if (lane == 0) wants[b] = missing;
       });
  const bool any_shared = __syncthreads_or(found_shared) != 0;
  if (any_shared) {
    walk([](int) {},
         [&](int entry, bool, int page, int held) {
           if (held > 1) {
             __hip_atomic_fetch_add(w.asks + page, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
             __hip_atomic_fetch_max(w.last + page, entry, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
           }
         },
         [](int) {});
    __syncthreads();
    int replaced = 0;
    walk([&](int) { replaced = 0; },
         [&](int entry, bool, int page, int held) {
           bool keeps = false;
           if (held > 1 && shared_load(w.last + page) == entry) {
             keeps = shared_load(w.asks + page) == held;
             // from here on: whether one of the others that ask got none; and no last one where none keeps the page
             shared_store(w.asks + page, 0);
             if (!keeps) shared_store(w.last + page, -1);
           }
           replaced += __popcll(__ballot(held > 1 && !keeps) & group);
         },
         [&](int b) {
           if (lane == 0) wants[b] += replaced;
         });
    __syncthreads();
  }
  int total = 0;
  for (int b0 = 0; b0 < d.sequences; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int sum;
    const int below = block_scan(b < d.sequences ? wants[b] : 0, sums, sum);
    if (b < d.sequences) w.rank[b] = wants[b] = total + below;
    total += sum;
  }
  // the first `total` free pages
  int found = 0;
  for (int64_t p0 = 0; p0 < d.pages && found < total; p0 += (int64_t)kPlanThreads * kPagesPerThread) {
    const int64_t first = p0 + (int64_t)tid * kPagesPerThread;
    uint32_t exist, open = used_pages(refs, first, d.pages, exist);
    open = exist & ~open;
    int sum;
    int rank = found + block_scan(__popc(open), sums, sum);
    for (; open != 0 && rank < total; open &= open - 1, ++rank) w.free[rank] = (int)first + __builtin_ctz(open);
    found += sum;
  }
  const int granted = min(found, total);
  if (tid == 0) *w.granted = granted;
  if (!any_shared || granted == total) return;
  // the pool ran out: who keeps a page that another one asked for in vain has it not to itself
  __syncthreads();
  int next = 0;
  walk([&](int b) { next = wants[b]; },
       [&](int entry, bool in, int page, int held) {
         const bool replaced = held > 1 && shared_load(w.last + page) != entry;
         const uint64_t all = __ballot((in && page < 0) || replaced) & group;
         if (replaced && next + __popcll(all & below_me) >= granted) shared_store(w.asks + page, 1);
         next += __popcll(all);
       },
       [](int) {});
}

// Rows 0 .. n - 1 of every head of page src into page dst, by the workgroups of blockIdx.y.
__device__ __forceinline__ void copy_rows(uint8_t* __restrict__ pool, int src, int dst, int64_t heads, int page_shift,
                                          int row_bytes, int n) {
  const int64_t head_bytes = (int64_t)row_bytes << page_shift, page_bytes = head_bytes * heads;
  const uint8_t* from = pool + src * page_bytes;
  uint8_t* to = pool + dst * page_bytes;
  const int bytes = n * row_bytes, chunks = (bytes + 15) / 16;
  for (int64_t i = (int64_t)blockIdx.y * kThreads + threadIdx.x; i < heads * chunks; i += (int64_t)gridDim.y * kThreads) {
    const int64_t head = i / chunks;
    const int at = (int)(i - head * chunks) * 16;
    const int64_t o = head * head_bytes + at;
    if (at + 16 <= bytes) *reinterpret_cast<u32x4_t*>(to + o) = *reinterpret_cast<const u32x4_t*>(from + o);
    else
      for (int k = 0; at + k < bytes; ++k) to[o + k] = from[o + k];
  }
}

__global__ void __launch_bounds__(kThreads) k_cache_reserve(CacheArgs c, const int32_t* __restrict__ table,
                                                            const int32_t* __restrict__ lengths,
                                                            const int32_t* __restrict__ refs,
                                                            const int32_t* __restrict__ tokens_each,
                                                            int32_t* __restrict__ table_out,
                                                            int32_t* __restrict__ refs_out, int32_t* __restrict__ short_out,
                                                            int32_t* __restrict__ work, ReserveDims d) {
  const ReserveSpace w = reserve_space(work, d.sequences, d.pages);
  const int b = blockIdx.x, granted = *w.granted;
  const int32_t* row = table + (int64_t)b * d.width;
  const Need n = need_of(lengths[b], tokens_each ? tokens_each[b] : d.tokens, d);
  const int rank = w.rank[b], filled = n.length & ((1 << d.page_shift) - 1);
  // the rows of a partly filled page that others name too, into the first page that the sequence gets
  if (n.slot < n.end && filled && rank < granted) {
    const int src = row[n.slot];
    if (valid_page(src, d.pages) && refs[src] > 1 && w.last[src] != b * d.width + n.slot) {
      const int dst = w.free[rank], codes = c.fmt == FMT_FP8 ? c.head_dim : c.head_dim / 2;
      copy_rows(c.k_codes, src, dst, c.kv_heads, d.page_shift, codes, filled);
      copy_rows(c.k_scales, src, dst, c.kv_heads, d.page_shift, c.head_dim / c.block, filled);
      if (!c.shared) {
        copy_rows(c.v_codes, src, dst, c.kv_heads, d.page_shift, codes, filled);
        copy_rows(c.v_scales, src, dst, c.kv_heads, d.page_shift, c.head_dim / c.block, filled);
      }
    }
  }
  if (blockIdx.y > 0 || threadIdx.x >= 64) return;
  // entries and counts: the first wave
  const int lane = threadIdx.x;
  int next = rank, lack = n.beyond;
  for (int s0 = n.slot; s0 < n.end; s0 += 64) {
    const int s = s0 + lane, entry = b * d.width + s;
    const bool in = s < n.end;
    int page = row[min(s, d.width - 1)];
    page = in && valid_page(page, d.pages) ? page : -1;
    const bool common = page >= 0 && refs[page] > 1, keeps = common && w.last[page] == entry;
    const bool want = in && (page < 0 || (common && !keeps));
    const uint64_t all = __ballot(want);
    const int mine = next + __popcll(all & ((1ull << lane) - 1));
    if (want && mine < granted) {
      const int fresh = w.free[mine];
      table_out[entry] = fresh;
      refs_out[fresh] = 1;
      if (page >= 0) atomicSub(refs_out + page, 1);
    }
    next += __popcll(all);
    lack += __popcll(__ballot((want && mine >= granted) || (keeps && w.asks[page])));
  }
  if (lane == 0) short_out[b] = lack;
}

// -------------------------------------------------------------------- accept
// A wave for each sequence, head and kind of row.  A place is never behind its
// row, and rows and places rise, so that a row moved later is no place of one
// moved before: rows go in groups, each group read before it is written.
__global__ void __launch_bounds__(64) k_cache_accept(CacheArgs c, const int32_t* __restrict__ table,
                                                     const int32_t* __restrict__ lengths,
                                                     const int32_t* __restrict__ refs,
                                                     const int32_t* __restrict__ accepted, int most, int width,
                                                     int page_shift, int32_t* __restrict__ lengths_out) {
  const int lane = threadIdx.x, b = blockIdx.x, head = blockIdx.y;
  const int length = cached_positions(lengths[b], width, 1 << page_shift);
  const int32_t* row = table + (int64_t)b * width;
  const int pick = lane < most ? accepted[(int64_t)b * most + lane] : -1;
  const int before = __shfl_up(pick, 1);
  bool good = pick >= 0 && (lane == 0 || pick > before);
  int src_page = -1, dst_page = -1;
  const int64_t src_pos = (int64_t)length + pick;
  if (good && src_pos < (int64_t)width << page_shift) {
    src_page = page_of(row, width, page_shift, c.pages, (int)src_pos);
    dst_page = page_of(row, width, page_shift, c.pages, length + lane);
  }
  good = src_page >= 0 && dst_page >= 0 && refs[max(dst_page, 0)] == 1;
  const uint64_t bad = ~__ballot(good);
  const int n = bad ? __builtin_ctzll(bad) : 64;
  if (head == 0 && blockIdx.z == 0 && lane == 0) lengths_out[b] = length + n;
  const int in_page = (1 << page_shift) - 1;
  const int64_t src = (((int64_t)src_page * c.kv_heads + head) << page_shift) + (src_pos & in_page);
  const int64_t dst = (((int64_t)dst_page * c.kv_heads + head) << page_shift) + ((length + lane) & in_page);
  uint8_t* codes = blockIdx.z ? c.v_codes : c.k_codes;
  uint8_t* scales = blockIdx.z ? c.v_scales : c.k_scales;
  const int code_chunks = (c.fmt == FMT_FP8 ? c.head_dim : c.head_dim / 2) / 16;   // 2 .. 32 lanes a row
  for (int a0 = 0; a0 < n; a0 += 64 / code_chunks) {
    const int a = a0 + lane / code_chunks;
    const int64_t from = __shfl(src, a & 63), to = __shfl(dst, a & 63);
    if (a < n && from != to) {
      const int64_t at = (lane % code_chunks) * 16;
      *reinterpret_cast<u32x4_t*>(codes + to * code_chunks * 16 + at) =
          *reinterpret_cast<const u32x4_t*>(codes + from * code_chunks * 16 + at);
    }
  }
  const int scale_bytes = c.head_dim / c.block;                                    // 1 .. 32 lanes a row
  for (int a0 = 0; a0 < n; a0 += 64 / scale_bytes) {
    const int a = a0 + lane / scale_bytes;
    const int64_t from = __shfl(src, a & 63), to = __shfl(dst, a & 63);
    if (a < n && from != to) scales[to * scale_bytes + lane % scale_bytes] = scales[from * scale_bytes + lane % scale_bytes];
  }
}

// ------------------------------------------------------------------- compact
// int32 arrays of the workspace: [0] used pages n, [1] pages that move, then the free pages below n, the used ones from n
// on (both rising), and where each of the latter goes.
struct CompactSpace {
  int32_t *head, *dst, *src, *to;
};
__host__ __device__ inline CompactSpace compact_space(int32_t* w, int64_t pages) {
  return {w, w + 2, w + 2 + (pages / 2 + 1), w + 2 + 2 * (pages / 2 + 1)};
}

__global__ void __launch_bounds__(kPlanThreads) k_cache_compact_plan(const int32_t* __restrict__ refs, int64_t pages,
                                                                     int32_t* __restrict__ work) {
  const CompactSpace w = compact_space(work, pages);
  const int tid = threadIdx.x;
  __shared__ int sums[kPlanWaves];
  const int64_t step = (int64_t)kPlanThreads * kPagesPerThread;
  int used = 0, n;
  for (int64_t p0 = 0; p0 < pages; p0 += step) {
    uint32_t exist;
    used += __popc(used_pages(refs, p0 + (int64_t)tid * kPagesPerThread, pages, exist));
  }
  block_scan(used, sums, n);
  int dst = 0, src = 0;
  for (int64_t p0 = 0; p0 < pages; p0 += step) {
    const int64_t first = p0 + (int64_t)tid * kPagesPerThread;
    uint32_t exist;
    const uint32_t use = used_pages(refs, first, pages, exist);
    const int64_t front = n - first;             // pages of this thread below n
    const uint32_t low = front >= kPagesPerThread ? 0xFFFFu : front <= 0 ? 0u : (1u << front) - 1;
    uint32_t open = exist & ~use & low, far = use & ~low;
    int sum;
    int rank = dst + block_scan(__popc(open), sums, sum);
    dst += sum;
    for (; open != 0; open &= open - 1, ++rank) w.dst[rank] = (int)first + __builtin_ctz(open);
    rank = src + block_scan(__popc(far), sums, sum);
    src += sum;
    for (; far != 0; far &= far - 1, ++rank) w.src[rank] = (int)first + __builtin_ctz(far);
  }
  __syncthreads();
  for (int i = tid; i < src; i += kPlanThreads) w.to[w.src[i]] = w.dst[i];
  if (tid == 0) {
    w.head[0] = n;
    w.head[1] = src;
  }
}

// Table and counts, then the pages that move: 16 KB of one pool's page at a time.
__global__ void __launch_bounds__(kThreads) k_cache_compact(CacheArgs c, const int32_t* __restrict__ table,
                                                            int64_t entries, const int32_t* __restrict__ refs,
                                                            int32_t* __restrict__ table_out,
                                                            int32_t* __restrict__ refs_out, int32_t* __restrict__ work) {
  const CompactSpace w = compact_space(work, c.pages);
  const int n = w.head[0], moved = w.head[1];
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = first; i < entries; i += step) {
    const int page = table[i];
    // an entry that names a page nobody counts has nowhere to go
    table_out[i] = !valid_page(page, c.pages) ? -1 : page < n ? page : refs[page] > 0 ? w.to[page] : -1;
  }
  for (int64_t p = first; p < c.pages; p += step)
    if (p >= n || refs[p] > 0) refs_out[p] = p < n ? refs[p] : 0;
  for (int64_t i = first; i < moved; i += step) refs_out[w.dst[i]] = refs[w.src[i]];
  const int64_t rows = (int64_t)c.kv_heads * c.page_size;
  const int64_t codes = rows * (c.fmt == FMT_FP8 ? c.head_dim : c.head_dim / 2), scales = rows * (c.head_dim / c.block);
  constexpr int64_t kPart = (int64_t)kThreads * 64;
  const int code_parts = (int)((codes + kPart - 1) / kPart), scale_parts = (int)((scales + kPart - 1) / kPart);
  const int parts = (code_parts + scale_parts) * (c.shared ? 1 : 2);
  for (int64_t u = blockIdx.x; u < (int64_t)moved * parts; u += gridDim.x) {
    const int pair = (int)(u / parts);
    int part = (int)(u - (int64_t)pair * parts);
    const bool second = part >= code_parts + scale_parts;
    if (second) part -= code_parts + scale_parts;
    const bool is_code = part < code_parts;
    uint8_t* pool = is_code ? (second ? c.v_codes : c.k_codes) : (second ? c.v_scales : c.k_scales);
    const int64_t bytes = is_code ? codes : scales, at = (int64_t)(is_code ? part : part - code_parts) * kPart;
    const uint8_t* from = pool + w.src[pair] * bytes;
    uint8_t* to = pool + w.dst[pair] * bytes;
    u32x4_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t o = at + ((int64_t)k * kThreads + threadIdx.x) * 16;
      if (o < bytes) v[k] = load16<true>(from + o);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t o = at + ((int64_t)k * kThreads + threadIdx.x) * 16;
      if (o < bytes) store16<true>(to + o, v[k]);
    }
  }
}

// Where one launch of cache_fork beats two: it spares 2.5 us here and 3.5 us on the host, and each counting workgroup takes
// 0.35 us for 1024 entries (1.4 thousand entries 3.0 us against 2.7 + 2.7, 33 thousand 12 against 2.7 + 2.7).
constexpr int64_t kOnceEntries = 8192, kOnceWorkgroups = 1024;

unsigned grid_of(int64_t items, int64_t each, int64_t most) {
  return (unsigned)max((int64_t)1, min((items + each - 1) / each, most));
}

}  // namespace

hipError_t launch_cache_fork(const TableArgs& t, int64_t pages, int page_size, const int32_t* parents, int children,
                             const int32_t* keep, bool release, int32_t* table_out, int32_t* lengths_out,
                             int32_t* refs_out, hipStream_t st) {
  const ForkDims d = {pages, t.sequences, children, t.width, log2_of(page_size), release};
  const ForkArgs a = {t.table, t.lengths, t.refs, parents, keep, table_out, lengths_out, refs_out};
  const int64_t added = (int64_t)children * t.width, gone = release ? (int64_t)t.sequences * t.width : 0;
  const int64_t counting = (pages + kOwnPages - 1) / kOwnPages;
  if (added + gone <= kOnceEntries && counting <= kOnceWorkgroups) {
    k_cache_fork_once<<<(unsigned)counting + grid_of(added, kPlanThreads, 64), kPlanThreads, 0, st>>>(a, d, (int)counting);
    return hipGetLastError();
  }
  k_cache_fork<<<grid_of(max(added, pages), kThreads, 4096), kThreads, 0, st>>>(a, d);
  if (added + gone > 0) k_cache_fork_count<<<grid_of(added + gone, kThreads, 4096), kThreads, 0, st>>>(a, d);
  return hipGetLastError();
}

int64_t reserve_workspace_bytes(int64_t sequences, int64_t width, int64_t pages) {
  return 4 * (1 + sequences + 2 * pages + min(pages, sequences * width));
}

hipError_t launch_cache_reserve(const CacheArgs& c, const TableArgs& t, int tokens, const int32_t* tokens_each,
                                int32_t* table_out, int32_t* refs_out, int32_t* short_out, int32_t* workspace,
                                hipStream_t st) {
  const ReserveDims d = {c.pages, t.sequences, t.width, log2_of(c.page_size), tokens};
  const int64_t items = max((int64_t)t.sequences * t.width, c.pages);
  k_cache_reserve_plan<<<1 + grid_of(items, kPlanThreads, 512), kPlanThreads, 0, st>>>(
      t.table, t.lengths, t.refs, tokens_each, table_out, refs_out, workspace, d);
  if (t.sequences > 0)
    k_cache_reserve<<<dim3(t.sequences, 8), kThreads, 0, st>>>(c, t.table, t.lengths, t.refs, tokens_each, table_out,
                                                               refs_out, short_out, workspace, d);
  return hipGetLastError();
}

hipError_t launch_cache_accept(const CacheArgs& c, const TableArgs& t, const int32_t* accepted, int most,
                               int32_t* lengths_out, hipStream_t st) {
  k_cache_accept<<<dim3(t.sequences, c.kv_heads, c.shared ? 1 : 2), 64, 0, st>>>(
      c, t.table, t.lengths, t.refs, accepted, most, t.width, log2_of(c.page_size), lengths_out);
  return hipGetLastError();
}

int64_t compact_workspace_bytes(int64_t pages) { return 4 * (2 + 2 * (pages / 2 + 1) + pages); }

hipError_t launch_cache_compact(const CacheArgs& c, const TableArgs& t, int32_t* table_out, int32_t* refs_out,
                                int32_t* workspace, hipStream_t st) {
  const int64_t entries = (int64_t)t.sequences * t.width;
  k_cache_compact_plan<<<1, kPlanThreads, 0, st>>>(t.refs, c.pages, workspace);
  k_cache_compact<<<2048, kThreads, 0, st>>>(c, t.table, entries, t.refs, table_out, refs_out, workspace);
  return hipGetLastError();
}

}  // namespace mxq
