// The grouped order of the routed slots and the rows' way there and back:
// moe_plan, moe_dispatch (plain and quantized), moe_combine and its gradient.
//
// moe_plan is a stable counting sort of n slots by local expert, bound by
// latency: its bytes are nothing.  A workgroup places 1024 slots at a time, one
// a thread.  A slot's row is the sum of four counts: the rows of lower experts,
// the expert's slots in earlier tiles, in earlier waves of this tile, and in
// lower lanes of this wave (the lanes with an equal expert, found bit by bit
// with ballots).  Up to kPlanRecount slots every workgroup counts all of them
// itself, which takes one launch; above, a first launch writes one histogram a
// tile.  Integer counts do not depend on the order of the LDS atomics.
//
// The row kernels are HBM streams.  A wave owns 64 chunks of 8 consecutive
// columns of one token, so the token's rows and weights are scalars, and visits
// its top_k rows: a token's row is read once (dispatch) or written once
// (combine) whatever top_k is, and the combine has the loads of 8 rows in
// flight.  Rows of the grouped order are read past the caches, and the
// combine's outputs and gradients written past them (they are top_k times what
// fits): bf16 [8192, 7168] x top-8, 1.06 GB, combine 203 -> 182 us and 173 with
// smaller workgroups (6.1 TB/s), its gradient, 2.0 GB, 391 -> 360 us (5.6 TB/s;
// 381 behind its forward).  The dispatch writes through the caches: its last rows
// are there for whoever reads them next.  Repeated alone it runs 197 us that way
// and 176 past the caches, but followed by its gradient the two take 371 us against
// 379.
#include "moe_launch.hpp"
#include "moe_device.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
// The combine reads top_k bytes for one that it writes; with half as large
// workgroups its read streams ran 5% faster (bf16 [8192, 7168] x top-8: 182 ->
// 173 us; 64 threads 175), where the dispatch measured the same and the
// quantized dispatch 1-5% slower.
constexpr int kCombineThreads = 128;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
// Every workgroup counting all slots against a launch of its own for the
// counts, 256 experts: 2048 slots 5.2 and 6.7 us, 16384 6.8 and 7.7, 32768 8.4 and
// 8.1, 131072 18.6 and 10.8.
constexpr int64_t kPlanRecount = 16384;
// Histograms that every workgroup of the second launch adds up: 524288 slots of
// 32 experts 17.7 us with 64, 12.0 with 128, 9.7 with 256 (of 256 experts 22.3,
// 16.6, 16.6).
constexpr int kPlanMaxTiles = 256;

// Buckets: the local experts, and one for the slots that are not served.
__device__ __forceinline__ int bucket_of(int expert, int first, int local) {
  const unsigned e = (unsigned)expert - (unsigned)first;
  return expert >= 0 && e < (unsigned)local ? (int)e : local;
}

// Lanes of the wave that hold the same bucket (of `bits` bits).
__device__ __forceinline__ uint64_t same_bucket(int b, int bits) {
  uint64_t m = ~0ull;
  for (int i = 0; i < bits; ++i) {
    const bool one = (b >> i) & 1;
    const uint64_t set = __ballot(one);
    m &= one ? set : ~set;
  }
  return m;
}

// Histogram of slots [lo, hi) into hist[local] (LDS); slots that are not served are not counted.
__device__ __forceinline__ void count_slots(const int32_t* __restrict__ index, int64_t lo, int64_t hi, int first,
                                            int local, int32_t* hist) {
  constexpr int kDeep = 4;             // loads in flight
  for (int64_t s0 = lo + threadIdx.x; s0 < hi; s0 += kDeep * kPlanThreads) {
    int32_t e[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) e[u] = s0 + u * kPlanThreads < hi ? index[s0 + u * kPlanThreads] : -1;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int b = bucket_of(e[u], first, local);
      if (b < local) atomicAdd(&hist[b], 1);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_moe_plan_count(const int32_t* __restrict__ index, int64_t n,
                                                                 int64_t tile, int first, int local,
                                                                 int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kMaxExperts];
  if ((int)threadIdx.x < local) hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * tile;
  count_slots(index, lo, min(n, lo + tile), first, local, hist);
  __syncthreads();
  if ((int)threadIdx.x < local) counts[(int64_t)blockIdx.x * local + threadIdx.x] = hist[threadIdx.x];
}

// COUNTED: counts holds a histogram a tile.  Slots [tile * block, tile * block + tile) are placed here.
template <bool COUNTED>
__global__ void __launch_bounds__(kPlanThreads) k_moe_plan_place(const int32_t* __restrict__ index, int64_t n,
                                                                 int64_t tile, int first, int local, int bits,
                                                                 const int32_t* __restrict__ counts,
                                                                 int32_t* __restrict__ offs, int32_t* __restrict__ rows,
                                                                 int32_t* __restrict__ slot_of_row) {
  __shared__ int32_t in_wave[kPlanWaves * (kMaxExperts + 1)];
  __shared__ int32_t before[kMaxExperts + 1], after[kMaxExperts];   // slots of an expert before this tile, and from it on
  __shared__ uint64_t part[kPlanWaves];
  const int nb = local + 1, b = threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = blockIdx.x * tile, t1 = min(n, t0 + tile);
  int64_t s = t0 + threadIdx.x;
  int32_t expert = s < t1 ? index[s] : -1;
  for (int i = threadIdx.x; i < kPlanWaves * nb; i += kPlanThreads) in_wave[i] = 0;
  if (b < local) before[b] = after[b] = 0;
  __syncthreads();
  if constexpr (COUNTED) {
    // threads of a bucket share its tiles
    const int parts = kPlanThreads / local, p = b / local, e = b - p * local;
    if (p < parts) {
      int32_t lo = 0, hi = 0;
#pragma unroll 4
      for (int w = p; w < (int)gridDim.x; w += parts) {
        const int32_t c = counts[(int64_t)w * local + e];
        lo += w < (int)blockIdx.x ? c : 0;
        hi += w < (int)blockIdx.x ? 0 : c;
      }
      atomicAdd(&before[e], lo);
      atomicAdd(&after[e], hi);
    }
  } else {
    count_slots(index, 0, t0, first, local, before);
    count_slots(index, t0, n, first, local, after);
  }
  __syncthreads();
  // exclusive scan over the experts of (all slots, slots before this tile), both below 2^31
  const uint64_t own = b < local ? ((uint64_t)(uint32_t)(before[b] + after[b]) << 32) | (uint32_t)before[b] : 0;
  uint64_t sum = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t u = __shfl_up(sum, d);
    if (lane >= d) sum += u;
  }
  if (lane == 63) part[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += part[w];
  if (b < local) {
    if (blockIdx.x == 0) offs[b] = (int32_t)(sum >> 32);
    before[b] += (int32_t)((sum - own) >> 32);
    // the slots that are not served follow the last expert's
    if (b == local - 1) before[local] = (int32_t)(sum >> 32) + (int32_t)(t0 - (int64_t)(uint32_t)sum);
  }
  for (;;) {
    const int mine = s < t1 ? bucket_of(expert, first, local) : nb;     // nb: no slot
    const uint64_t same = same_bucket(mine, bits);
    const int lower = __popcll(same & ((1ull << lane) - 1));
    if (s < t1 && lower == 0) in_wave[wave * nb + mine] = __popcll(same);
    __syncthreads();
    if (s < t1) {
      int r = before[mine] + lower;
      for (int w = 0; w < wave; ++w) r += in_wave[w * nb + mine];
      rows[s] = mine < local ? r : ~r;
      if ((uint64_t)(int64_t)r < (uint64_t)n) slot_of_row[r] = (int32_t)s;   // always, unless index changed meanwhile
    }
    if (s - threadIdx.x + kPlanThreads >= t1) break;                    // the same for the whole workgroup
    s += kPlanThreads;
    expert = s < t1 ? index[s] : -1;
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kPlanThreads) {              // these slots lie before the next 1024
      int c = 0;
      for (int w = 0; w < kPlanWaves; ++w) {
        c += in_wave[w * nb + i];
        in_wave[w * nb + i] = 0;
      }
      before[i] += c;
    }
    __syncthreads();
  }
}

int64_t plan_tile(int64_t n) {
  if (n <= kPlanRecount) return kPlanThreads;
  const int64_t t = (n + kPlanMaxTiles - 1) / kPlanMaxTiles;
  return (t + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

// ------------------------------------------------------------- row streams
constexpr int kDeep = 8;               // rows in flight

// The token and the chunk of 8 columns of this lane: 64 consecutive chunks of
// one token a wave, `segs` waves a token.
struct Place {
  int64_t token;
  int chunk;
};
template <int THREADS>
__device__ __forceinline__ Place place_of(unsigned segs) {
  const unsigned w = blockIdx.x * (THREADS / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned token = w / segs;
  return {token, (int)((w - token * segs) * 64 + (threadIdx.x & 63))};
}

// Columns of a chunk.  The last chunk of a row whose width is no multiple of 8
// is moved back to end with the row: it repeats the columns that it shares with
// the chunk before it (the same values, so both may be written), and every
// access takes 16 bytes.  NARROW rows (under 8 columns) have one chunk, of
// `live` columns.
struct Columns {
  int64_t first;
  int live, repeated;
};
template <bool NARROW>
__device__ __forceinline__ Columns columns_of(int chunk, int64_t hidden) {
  const int64_t at = (int64_t)chunk * 8;
  if constexpr (NARROW) return {at, (int)hidden, 0};
  const int64_t first = min(at, hidden - 8);
  return {first, 8, (int)(at - first)};
}

// The row that a value of `rows` names, or -1.  served: whether it belongs to an expert.
__device__ __forceinline__ int64_t row_of(int32_t v, int64_t n, bool& served) {
  served = v >= 0;
  const int64_t r = served ? v : ~v;
  return r < n ? r : -1;
}

template <int DT, bool NARROW>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch(const uint8_t* __restrict__ x, int64_t tokens, int64_t hidden,
                                                           int chunks, unsigned segs, int top_k,
                                                           const int32_t* __restrict__ rows,
                                                           uint8_t* __restrict__ out) {
  const Place p = place_of<kThreads>(segs);
  if (p.token >= tokens || p.chunk >= chunks) return;
  const Columns c = columns_of<NARROW>(p.chunk, hidden);
  const int64_t rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  const Raw8<DT> v = load8<DT>(x + p.token * rb, c.first, c.live);
  for (int j = 0; j < top_k; ++j) {
    bool served;
    const int64_t r = row_of(rows[p.token * top_k + j], n, served);
    if (r >= 0) store8<DT>(out + r * rb, c.first, c.live, served ? v : zero8<DT>());
  }
}

// Four lanes hold a block of 32 columns.
template <int DT, bool FP4>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch_quantized(const uint8_t* __restrict__ x, int64_t tokens,
                                                                     int64_t hidden, int chunks, unsigned segs,
                                                                     int top_k, const int32_t* __restrict__ rows,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  const Place p = place_of<kThreads>(segs);
  if (p.token >= tokens || p.chunk >= chunks) return;   // whole groups of four lanes: chunks is a multiple of 4
  float v[8];
  to_f32<DT>(load8<DT>(x + p.token * hidden * kElemBytes<DT>, (int64_t)p.chunk * 8, 8), v);
  const uint32_t amax = group_max_u32<4>(amax_bits(v));
  const int k = FP4 ? floor_rule_exponent(amax) : ceil_rule_exponent<FMT_FP8>(amax);
  const int none = FP4 ? floor_rule_exponent(0u) : ceil_rule_exponent<FMT_FP8>(0u);
  u32x2_t c = {0u, 0u};
  if constexpr (FP4) c.x = encode_fp4(v, pow2f(k));
  else c = encode_fp8(v, pow2f(k));
  const uint32_t bytes = scale_bytes(k, p.chunk);
  const bool whole = (p.chunk | 15) < chunks;          // the same for 16 lanes
  const int64_t n = tokens * top_k;
  for (int j = 0; j < top_k; ++j) {
    bool served;
    const int64_t r = row_of(rows[p.token * top_k + j], n, served);
    if (r < 0) continue;
    const int64_t at = r * chunks + p.chunk;
    if constexpr (FP4) store4<true>(codes + at * 4, served ? c.x : 0u);
    else store_8<true>(codes + at * 8, served ? c : u32x2_t{0u, 0u});
    const uint32_t sb = served ? bytes : (uint32_t)(none + 127) * 0x01010101u;
    if (whole) {
      if ((p.chunk & 15) == 0) store4<false>(scales + (at >> 2), sb);
    } else if ((p.chunk & 3) == 0) {
      scales[at >> 2] = (uint8_t)(sb >> (8 * ((p.chunk >> 2) & 3)));
    }
  }
}

// WEIGHTED false: weights of 1.  A slot that is not served, and a place past top_k
// in a round of 8, reads row 0 and adds nothing of it, so that every lane has the
// same 8 loads in flight.  That is made for top_k of 8 with every expert here; off
// that the idle loads show: bf16 [8192, 7168], top-1 81 us (its bytes take 29 at 8
// TB/s), top-4 104 (73), top-8 175 (132), top-9 203 (147), top-8 with a quarter of
// the experts here 79 (44).  k_moe_combine_bwd loads alike: 117 (44), 198 (132), 360
// (250), 432 (279), 293 (161).
template <int DT, bool WEIGHTED, bool NARROW>
__global__ void __launch_bounds__(kCombineThreads) k_moe_combine(const uint8_t* __restrict__ y, int64_t tokens, int64_t hidden,
                                                          int chunks, unsigned segs, int top_k,
                                                          const int32_t* __restrict__ rows,
                                                          const float* __restrict__ weights,
                                                          uint8_t* __restrict__ out) {
  const Place p = place_of<kCombineThreads>(segs);
  if (p.token >= tokens || p.chunk >= chunks) return;
  const Columns c = columns_of<NARROW>(p.chunk, hidden);
  const int64_t rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  float acc[8] = {};
  for (int j0 = 0; j0 < top_k; j0 += kDeep) {
    Raw8<DT> raw[kDeep];
    bool use[kDeep];
    float w[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int64_t slot = p.token * top_k + min(j0 + u, top_k - 1);
      bool served;
      const int64_t r = row_of(rows[slot], n, served);
      use[u] = served && r >= 0 && j0 + u < top_k;
      w[u] = WEIGHTED ? weights[slot] : 1.0f;
      raw[u] = load8<DT, true>(y + (use[u] ? r : 0) * rb, c.first, c.live);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (!use[u]) continue;
      float v[8];
      to_f32<DT>(raw[u], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[u], v[i], acc[i]);
    }
  }
  store8<DT, true>(out + p.token * rb, c.first, c.live, from_f32<DT>(acc));
}

// One workgroup per token, 8 slots at a time: a lane reads its chunk of
// grad_out once for the 8, and keeps 8 partial dots, which go lane -> wave ->
// workgroup in a fixed order.
constexpr int kBwdWaves = 8;
template <int DT, bool GY, bool GW, bool NARROW>
__global__ void __launch_bounds__(kBwdWaves * 64) k_moe_combine_bwd(const uint8_t* __restrict__ grad_out,
                                                                    const uint8_t* __restrict__ y, int64_t tokens,
                                                                    int64_t hidden, int chunks, int top_k,
                                                                    const int32_t* __restrict__ rows,
                                                                    const float* __restrict__ weights,
                                                                    uint8_t* __restrict__ grad_y,
                                                                    float* __restrict__ grad_weights) {
  __shared__ float dots[kDeep][kBwdWaves];
  const int64_t token = blockIdx.x, rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int j0 = 0; j0 < top_k; j0 += kDeep) {
    int64_t r[kDeep];
    bool served[kDeep];
    float w[kDeep], dot[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int64_t slot = token * top_k + min(j0 + u, top_k - 1);
      r[u] = row_of(rows[slot], n, served[u]);
      served[u] = served[u] && r[u] >= 0 && j0 + u < top_k;
      if (j0 + u >= top_k) r[u] = -1;
      w[u] = GY && served[u] ? weights[slot] : 0.0f;
      dot[u] = 0.0f;
    }
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      const Columns at = columns_of<NARROW>(c, hidden);
      Raw8<DT> raw[kDeep];
      float g[8];
      if constexpr (GW) {
#pragma unroll
        for (int u = 0; u < kDeep; ++u) raw[u] = load8<DT, true>(y + (served[u] ? r[u] : 0) * rb, at.first, at.live);
      }
      to_f32<DT>(load8<DT>(grad_out + token * rb, at.first, at.live), g);
      float once[8];                   // g where this chunk's columns count for the dots
#pragma unroll
      for (int i = 0; i < 8; ++i) once[i] = i < at.repeated ? 0.0f : g[i];
      if constexpr (GW && !NARROW) {
        if (at.repeated > 0) {         // y's too: 0 times an infinity is no 0
#pragma unroll
          for (int u = 0; u < kDeep; ++u) clear_first<DT>(raw[u], at.repeated);
        }
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        float v[8];
        if constexpr (GW) {
          if (served[u]) {
            to_f32<DT>(raw[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[u] = __builtin_fmaf(once[i], v[i], dot[u]);
          }
        }
        if constexpr (GY) {
          if (r[u] >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[u] * g[i];
            store8<DT, true>(grad_y + r[u] * rb, at.first, at.live, served[u] ? from_f32<DT>(v) : zero8<DT>());
          }
        }
      }
    }
    if constexpr (GW) {
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        float d = dot[u];
#pragma unroll
        for (int i = 32; i > 0; i >>= 1) d += __shfl_xor(d, i);
        if (lane == 0) dots[u][wave] = d;
      }
      __syncthreads();
      if ((int)threadIdx.x < min(kDeep, top_k - j0)) {
        float s = 0.0f;
        for (int i = 0; i < waves; ++i) s += dots[threadIdx.x][i];
        grad_weights[token * top_k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// Waves a token of the row streams, and their workgroups (0: more than a launch takes).
unsigned segs_of(int chunks) { return (unsigned)(chunks + 63) / 64; }
unsigned stream_blocks(int64_t tokens, int chunks, int threads) {
  const int64_t per = threads / 64, blocks = (tokens * segs_of(chunks) + per - 1) / per;
  return launchable(blocks, threads) ? (unsigned)blocks : 0u;
}

}  // namespace

int64_t plan_workspace_bytes(int64_t slots, int local) {
  if (slots <= kPlanRecount) return 0;
  const int64_t tile = plan_tile(slots);
  return (slots + tile - 1) / tile * local * 4;
}

hipError_t launch_moe_plan(const int32_t* index, int64_t slots, int first, int local, int32_t* offs, int32_t* rows,
                           int32_t* slot_of_row, int32_t* workspace, hipStream_t st) {
  const int64_t tile = plan_tile(slots);
  const int tiles = (int)max((int64_t)1, (slots + tile - 1) / tile);
  int bits = 1;                        // of the buckets 0 .. local, and local + 1 for lanes without a slot
  while ((1 << bits) <= local + 1) ++bits;
  if (slots <= kPlanRecount) {
    k_moe_plan_place<false><<<tiles, kPlanThreads, 0, st>>>(index, slots, tile, first, local, bits, nullptr, offs, rows,
                                                            slot_of_row);
    return hipGetLastError();
  }
  k_moe_plan_count<<<tiles, kPlanThreads, 0, st>>>(index, slots, tile, first, local, workspace);
  k_moe_plan_place<true><<<tiles, kPlanThreads, 0, st>>>(index, slots, tile, first, local, bits, workspace, offs, rows,
                                                         slot_of_row);
  return hipGetLastError();
}

#define MXQ_BY_DTYPE(dt, CALL)                   \
  do {                                           \
    if ((dt) == DT_F32) { CALL(DT_F32); }        \
    else if ((dt) == DT_BF16) { CALL(DT_BF16); } \
    else { CALL(DT_F16); }                       \
  } while (0)

hipError_t launch_moe_dispatch(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                               void* out, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  const unsigned blocks = stream_blocks(tokens, chunks, kThreads), segs = segs_of(chunks);
  if (blocks == 0) return hipErrorInvalidValue;
#define LAUNCH(DT, NARROW)                                                                                          \
  k_moe_dispatch<DT, NARROW><<<blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden, chunks, segs, top_k, \
                                                          rows, (uint8_t*)out)
#define CALL(DT)                      \
  if (hidden < 8) LAUNCH(DT, true);   \
  else LAUNCH(DT, false)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
#undef LAUNCH
  return hipGetLastError();
}

hipError_t launch_moe_dispatch_quantized(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k,
                                         const int32_t* rows, int fmt, uint8_t* codes, uint8_t* scales,
                                         hipStream_t st) {
  const int chunks = (int)(hidden / 8);
  const unsigned blocks = stream_blocks(tokens, chunks, kThreads), segs = segs_of(chunks);
  if (blocks == 0) return hipErrorInvalidValue;
#define CALL(DT)                                                                                                    \
  if (fmt == FMT_MXFP4)                                                                                             \
    k_moe_dispatch_quantized<DT, true><<<blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden,   \
                                                                              chunks, segs, top_k, rows, codes, scales);  \
  else                                                                                                              \
    k_moe_dispatch_quantized<DT, false><<<blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden,  \
                                                                               chunks, segs, top_k, rows, codes, scales)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                              const float* weights, void* out, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  const unsigned blocks = stream_blocks(tokens, chunks, kCombineThreads), segs = segs_of(chunks);
  if (blocks == 0) return hipErrorInvalidValue;
#define LAUNCH(DT, WEIGHTED, NARROW)                                                                              \
  k_moe_combine<DT, WEIGHTED, NARROW><<<blocks, kCombineThreads, 0, st>>>((const uint8_t*)y, tokens, hidden, chunks,    \
                                                                   segs, top_k, rows, weights, (uint8_t*)out)
#define CALL(DT)                                        \
  if (hidden < 8) {                                     \
    if (weights) LAUNCH(DT, true, true);                \
    else LAUNCH(DT, false, true);                       \
  } else if (weights) LAUNCH(DT, true, false);          \
  else LAUNCH(DT, false, false)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
#undef LAUNCH
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* grad_out, const void* y, int dt, int64_t tokens, int64_t hidden,
                                  int top_k, const int32_t* rows, const float* weights, void* grad_y,
                                  float* grad_weights, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  // waves of a workgroup: as few rounds over the columns as 8 waves give, and no idle wave in the last
  const int segs = max(1, (int)segs_of(chunks)), rounds = (segs + kBwdWaves - 1) / kBwdWaves;
  const unsigned threads = 64u * ((segs + rounds - 1) / rounds);
  if (!launchable(tokens, threads)) return hipErrorInvalidValue;
#define LAUNCH(DT, GY, GW, NARROW)                                                                                \
  k_moe_combine_bwd<DT, GY, GW, NARROW><<<(unsigned)tokens, threads, 0, st>>>(                                   \
      (const uint8_t*)grad_out, (const uint8_t*)y, tokens, hidden, chunks, top_k, rows, weights, (uint8_t*)grad_y, \
      grad_weights)
#define WANTED(DT, NARROW)                                        \
  if (grad_y && grad_weights) LAUNCH(DT, true, true, NARROW);     \
  else if (grad_y) LAUNCH(DT, true, false, NARROW);               \
  else LAUNCH(DT, false, true, NARROW)
#define CALL(DT)                          \
  if (hidden < 8) { WANTED(DT, true); }   \
  else { WANTED(DT, false); }
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
#undef WANTED
#undef LAUNCH
  return hipGetLastError();
}

}  // namespace mxq
