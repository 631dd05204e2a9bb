// The grouped order of the routed slots and the rows' way there and back:
// moe_plan, moe_dispatch (plain and quantized), moe_combine and its gradient.
//
// moe_plan is a stable counting sort of n slots by local expert, without
// atomics on the result: a wave owns a contiguous run of slots, so an
// exclusive scan over (expert, wave) of the waves' histograms gives every
// wave its first row per expert, and inside 64 slots a slot's place among
// equal experts is the number of lower lanes that hold the same expert.
//
// The row kernels are HBM streams.  A lane owns a chunk of 8 consecutive
// elements of one token and visits the token's top_k rows, so a token's row is
// read once (dispatch) or written once (combine) whatever top_k is.
#include "moe_launch.hpp"
#include "moe_device.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
// Slots that one workgroup sorts by itself; more are cut into tiles.
constexpr int64_t kPlanOneSlots = 16384;
constexpr int64_t kPlanTile = 4096;
constexpr int kPlanMaxTiles = 256;

// Buckets: the local experts, and one for the slots that are not served.
__device__ __forceinline__ int bucket_of(int expert, int first, int local) {
  const unsigned e = (unsigned)expert - (unsigned)first;
  return expert >= 0 && e < (unsigned)local ? (int)e : local;
}

// Lanes of the wave that hold the same bucket (bits < 11), among the active ones.
__device__ __forceinline__ uint64_t same_bucket(int b, uint64_t active) {
  uint64_t m = active;
#pragma unroll
  for (int i = 0; i < 11; ++i) {
    const uint64_t set = __ballot((b >> i) & 1);
    m &= (b >> i) & 1 ? set : ~set;
  }
  return m;
}

// Histogram of slots [lo, hi) into hist[local + 1] by the lanes of one wave.
__device__ __forceinline__ void wave_histogram(const int32_t* __restrict__ index, int64_t lo, int64_t hi, int first,
                                               int local, int32_t* hist) {
  const int lane = threadIdx.x & 63;
  for (int64_t s = lo + lane; s < hi; s += 64) atomicAdd(&hist[bucket_of(index[s], first, local)], 1);
}

// Rows of slots [lo, hi), 64 at a time; next[b] is the wave's next row of bucket b.
__device__ __forceinline__ void wave_place(const int32_t* __restrict__ index, int64_t lo, int64_t hi, int first,
                                           int local, int32_t* next, int32_t* __restrict__ rows,
                                           int32_t* __restrict__ slot_of_row) {
  const int lane = threadIdx.x & 63;
  for (int64_t s0 = lo; s0 < hi; s0 += 64) {
    const int64_t s = s0 + lane;
    const bool on = s < hi;
    const int b = on ? bucket_of(index[s], first, local) : 0x7FF;
    const uint64_t same = same_bucket(b, __ballot(on));
    const int before = __popcll(same & ((1ull << lane) - 1));
    if (on) {
      const int r = next[b] + before;
      rows[s] = b < local ? r : ~r;
      slot_of_row[r] = (int32_t)s;
    }
    wave_sync();                       // every lane has read next
    if (on && before == 0) next[b] += __popcll(same);
    wave_sync();
  }
}

// Exclusive scan over buckets of `total` (one int per thread, bucket = thread), in LDS; returns this thread's start.
__device__ __forceinline__ int block_exclusive_scan(int total, int32_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int v = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  if (lane == 63) part[wave] = v;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += part[w];
  return before + v - total;
}

// One workgroup: hist [waves][local + 1] in LDS.  local + 1 <= 1025 buckets:
// the first 1024 are scanned one per thread and the last starts where they end.
__global__ void __launch_bounds__(kPlanThreads) k_moe_plan_one(const int32_t* __restrict__ index, int64_t n, int first,
                                                               int local, int32_t* __restrict__ offs,
                                                               int32_t* __restrict__ rows,
                                                               int32_t* __restrict__ slot_of_row) {
  __shared__ int32_t hist[kPlanWaves * (kMaxExperts + 1)];
  __shared__ int32_t part[kPlanWaves];
  const int nb = local + 1, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kPlanWaves * nb; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int64_t run = (n + kPlanThreads - 1) / kPlanThreads * 64;   // slots of a wave
  const int64_t lo = min(n, wave * run), hi = min(n, lo + run);
  wave_histogram(index, lo, hi, first, local, hist + wave * nb);
  __syncthreads();
  const int b = threadIdx.x;
  int total = 0;
  if (b < local)
    for (int w = 0; w < kPlanWaves; ++w) total += hist[w * nb + b];
  int at = block_exclusive_scan(total, part);
  if (b < local) {
    offs[b] = at + total;
    if (b == local - 1) {              // the slots that are not served follow the last expert
      int rest = at + total;
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = hist[w * nb + local];
        hist[w * nb + local] = rest;
        rest += c;
      }
    }
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * nb + b];
      hist[w * nb + b] = at;
      at += c;
    }
  }
  __syncthreads();
  wave_place(index, lo, hi, first, local, hist + wave * nb, rows, slot_of_row);
}

// Many workgroups: a histogram per tile, then every tile adds up what lies before it.
__global__ void __launch_bounds__(kPlanThreads) k_moe_plan_count(const int32_t* __restrict__ index, int64_t n,
                                                                 int64_t tile, int first, int local,
                                                                 int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kMaxExperts + 1];
  const int nb = local + 1;
  for (int i = threadIdx.x; i < nb; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * tile, hi = min(n, lo + tile);
  for (int64_t s = lo + threadIdx.x; s < hi; s += kPlanThreads) atomicAdd(&hist[bucket_of(index[s], first, local)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < nb; i += kPlanThreads) counts[(int64_t)blockIdx.x * nb + i] = hist[i];
}

__global__ void __launch_bounds__(kPlanThreads) k_moe_plan_place(const int32_t* __restrict__ index, int64_t n,
                                                                 int64_t tile, int first, int local,
                                                                 const int32_t* __restrict__ counts,
                                                                 int32_t* __restrict__ offs, int32_t* __restrict__ rows,
                                                                 int32_t* __restrict__ slot_of_row) {
  __shared__ int32_t hist[kPlanWaves * (kMaxExperts + 1)];
  __shared__ int32_t part[kPlanWaves];
  __shared__ int32_t rest_before;
  const int nb = local + 1, wave = threadIdx.x >> 6, me = blockIdx.x, tiles = gridDim.x;
  for (int i = threadIdx.x; i < kPlanWaves * nb; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int64_t t0 = me * tile, t1 = min(n, t0 + tile);
  const int64_t run = (tile + kPlanThreads - 1) / kPlanThreads * 64;
  const int64_t lo = min(t1, t0 + wave * run), hi = min(t1, lo + run);
  wave_histogram(index, lo, hi, first, local, hist + wave * nb);
  const int b = threadIdx.x;
  int total = 0, before = 0;
  if (b < local)
    for (int w = 0; w < tiles; ++w) {
      const int c = counts[(int64_t)w * nb + b];
      total += c;
      before += w < me ? c : 0;
    }
  if (b == 0) {
    int r = 0;
    for (int w = 0; w < me; ++w) r += counts[(int64_t)w * nb + local];
    rest_before = r;
  }
  __syncthreads();
  const int start = block_exclusive_scan(total, part);
  if (b < local) {
    if (me == 0) offs[b] = start + total;
    int at = start + before;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * nb + b];
      hist[w * nb + b] = at;
      at += c;
    }
    if (b == local - 1) {
      int rest = start + total + rest_before;
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = hist[w * nb + local];
        hist[w * nb + local] = rest;
        rest += c;
      }
    }
  }
  __syncthreads();
  wave_place(index, lo, hi, first, local, hist + wave * nb, rows, slot_of_row);
}

int64_t plan_tile(int64_t n) {
  const int64_t t = (n + kPlanMaxTiles - 1) / kPlanMaxTiles;
  return max(kPlanTile, (t + kPlanThreads - 1) / kPlanThreads * kPlanThreads);
}

// ------------------------------------------------------------- row streams
// Chunk c of the flat list tokens x chunks-per-token that this lane owns.
struct Place {
  int64_t token;
  int chunk;
};
__device__ __forceinline__ Place place_of(int chunks) {
  const int64_t base = (int64_t)blockIdx.x * kThreads;
  const int64_t t0 = base / chunks;
  const unsigned at = (unsigned)(base - t0 * chunks) + threadIdx.x;
  const unsigned dt = at / (unsigned)chunks;
  return {t0 + dt, (int)(at - dt * (unsigned)chunks)};
}

// The row that a value of `rows` names, or -1.  served: whether it belongs to an expert.
__device__ __forceinline__ int64_t row_of(int32_t v, int64_t n, bool& served) {
  served = v >= 0;
  const int64_t r = served ? v : ~v;
  return r < n ? r : -1;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch(const uint8_t* __restrict__ x, int64_t tokens, int64_t hidden,
                                                           int chunks, int top_k, const int32_t* __restrict__ rows,
                                                           uint8_t* __restrict__ out) {
  const Place p = place_of(chunks);
  if (p.token >= tokens) return;
  const int64_t e = (int64_t)p.chunk * 8, rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  const int live = (int)min((int64_t)8, hidden - e);
  const Raw8<DT> v = load8<DT>(x + p.token * rb, e, live);
  for (int j = 0; j < top_k; ++j) {
    bool served;
    const int64_t r = row_of(rows[p.token * top_k + j], n, served);
    if (r >= 0) store8<DT>(out + r * rb, e, live, served ? v : zero8<DT>());
  }
}

// Four lanes hold a block of 32 columns.
template <int DT, bool FP4>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch_quantized(const uint8_t* __restrict__ x, int64_t tokens,
                                                                     int64_t hidden, int chunks, int top_k,
                                                                     const int32_t* __restrict__ rows,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  const Place p = place_of(chunks);
  if (p.token >= tokens) return;       // whole groups of four lanes: chunks is a multiple of 4
  float v[8];
  to_f32<DT>(load8<DT>(x + p.token * hidden * kElemBytes<DT>, (int64_t)p.chunk * 8, 8), v);
  const uint32_t amax = group_max_u32<4>(amax_bits(v));
  const int k = FP4 ? floor_rule_exponent(amax) : ceil_rule_exponent<FMT_FP8>(amax);
  const int none = FP4 ? floor_rule_exponent(0u) : ceil_rule_exponent<FMT_FP8>(0u);
  u32x2_t c = {0u, 0u};
  if constexpr (FP4) c.x = encode_fp4(v, pow2f(k));
  else c = encode_fp8(v, pow2f(k));
  const int64_t n = tokens * top_k;
  for (int j = 0; j < top_k; ++j) {
    bool served;
    const int64_t r = row_of(rows[p.token * top_k + j], n, served);
    if (r < 0) continue;
    if constexpr (FP4) *reinterpret_cast<u32_any*>(codes + (r * chunks + p.chunk) * 4) = served ? c.x : 0u;
    else *reinterpret_cast<u32x2_any*>(codes + (r * chunks + p.chunk) * 8) = served ? c : u32x2_t{0u, 0u};
    if ((p.chunk & 3) == 0) scales[(r * chunks + p.chunk) >> 2] = (uint8_t)((served ? k : none) + 127);
  }
}

// WEIGHTED false: weights of 1.
template <int DT, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) k_moe_combine(const uint8_t* __restrict__ y, int64_t tokens, int64_t hidden,
                                                          int chunks, int top_k, const int32_t* __restrict__ rows,
                                                          const float* __restrict__ weights,
                                                          uint8_t* __restrict__ out) {
  const Place p = place_of(chunks);
  if (p.token >= tokens) return;
  const int64_t e = (int64_t)p.chunk * 8, rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  const int live = (int)min((int64_t)8, hidden - e);
  float acc[8] = {};
  for (int j = 0; j < top_k; ++j) {
    bool served;
    const int64_t r = row_of(rows[p.token * top_k + j], n, served);
    if (r < 0 || !served) continue;
    const float w = WEIGHTED ? weights[p.token * top_k + j] : 1.0f;
    float v[8];
    to_f32<DT>(load8<DT>(y + r * rb, e, live), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
  }
  store8<DT>(out + p.token * rb, e, live, from_f32<DT>(acc));
}

// One workgroup per token: a lane keeps its chunks of grad_out for all slots
// by reading them again from the caches; dots go lane -> wave -> workgroup in
// a fixed order.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_moe_combine_bwd(const uint8_t* __restrict__ grad_out,
                                                              const uint8_t* __restrict__ y, int64_t tokens,
                                                              int64_t hidden, int chunks, int top_k,
                                                              const int32_t* __restrict__ rows,
                                                              const float* __restrict__ weights,
                                                              uint8_t* __restrict__ grad_y,
                                                              float* __restrict__ grad_weights) {
  __shared__ float dots[kMaxTopK][kThreads / 64];
  const int64_t token = blockIdx.x, rb = hidden * kElemBytes<DT>, n = tokens * top_k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < top_k; j0 += kMaxTopK) {
    const int jn = min(kMaxTopK, top_k - j0);
    for (int j = 0; j < jn; ++j) {
      const int64_t slot = token * top_k + j0 + j;
      bool served;
      const int64_t r = row_of(rows[slot], n, served);
      float dot = 0.0f;
      if (r >= 0) {
        const float w = served && grad_y ? weights[slot] : 0.0f;
        for (int c = threadIdx.x; c < chunks; c += kThreads) {
          const int64_t e = (int64_t)c * 8;
          const int live = (int)min((int64_t)8, hidden - e);
          float g[8], v[8];
          to_f32<DT>(load8<DT>(grad_out + token * rb, e, live), g);
          if (grad_weights && served) {
            to_f32<DT>(load8<DT>(y + r * rb, e, live), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(g[i], v[i], dot);
          }
          if (grad_y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = served ? w * g[i] : 0.0f;
            store8<DT>(grad_y + r * rb, e, live, from_f32<DT>(v));
          }
        }
      }
      if (grad_weights) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) dots[j][wave] = dot;
      }
    }
    if (grad_weights) {
      __syncthreads();
      if ((int)threadIdx.x < jn) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) s += dots[threadIdx.x][w];
        grad_weights[token * top_k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

int64_t flat_blocks(int64_t tokens, int64_t chunks) { return (tokens * chunks + kThreads - 1) / kThreads; }

}  // namespace

int64_t plan_workspace_bytes(int64_t slots, int local) {
  if (slots <= kPlanOneSlots) return 0;
  const int64_t tile = plan_tile(slots);
  return (slots + tile - 1) / tile * (local + 1) * 4;
}

hipError_t launch_moe_plan(const int32_t* index, int64_t slots, int first, int local, int32_t* offs, int32_t* rows,
                           int32_t* slot_of_row, int32_t* workspace, hipStream_t st) {
  if (slots <= kPlanOneSlots) {
    k_moe_plan_one<<<1, kPlanThreads, 0, st>>>(index, slots, first, local, offs, rows, slot_of_row);
    return hipGetLastError();
  }
  const int64_t tile = plan_tile(slots);
  const int tiles = (int)((slots + tile - 1) / tile);
  k_moe_plan_count<<<tiles, kPlanThreads, 0, st>>>(index, slots, tile, first, local, workspace);
  k_moe_plan_place<<<tiles, kPlanThreads, 0, st>>>(index, slots, tile, first, local, workspace, offs, rows,
                                                     slot_of_row);
  return hipGetLastError();
}

#define MXQ_BY_DTYPE(dt, CALL)                 \
  do {                                         \
    if ((dt) == DT_F32) { CALL(DT_F32); }      \
    else if ((dt) == DT_BF16) { CALL(DT_BF16); } \
    else { CALL(DT_F16); }                     \
  } while (0)

hipError_t launch_moe_dispatch(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                               void* out, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  const int64_t blocks = flat_blocks(tokens, chunks);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
#define CALL(DT)                                                                                                     \
  k_moe_dispatch<DT><<<(unsigned)blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden, chunks, top_k, rows, \
                                                            (uint8_t*)out)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_moe_dispatch_quantized(const void* x, int dt, int64_t tokens, int64_t hidden, int top_k,
                                         const int32_t* rows, int fmt, uint8_t* codes, uint8_t* scales,
                                         hipStream_t st) {
  const int chunks = (int)(hidden / 8);
  const int64_t blocks = flat_blocks(tokens, chunks);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
#define CALL(DT)                                                                                                    \
  if (fmt == FMT_MXFP4)                                                                                             \
    k_moe_dispatch_quantized<DT, true><<<(unsigned)blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden,   \
                                                                              chunks, top_k, rows, codes, scales);  \
  else                                                                                                              \
    k_moe_dispatch_quantized<DT, false><<<(unsigned)blocks, kThreads, 0, st>>>((const uint8_t*)x, tokens, hidden,  \
                                                                               chunks, top_k, rows, codes, scales)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int dt, int64_t tokens, int64_t hidden, int top_k, const int32_t* rows,
                              const float* weights, void* out, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  const int64_t blocks = flat_blocks(tokens, chunks);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
#define CALL(DT)                                                                                                   \
  if (weights)                                                                                                     \
    k_moe_combine<DT, true><<<(unsigned)blocks, kThreads, 0, st>>>((const uint8_t*)y, tokens, hidden, chunks,      \
                                                                   top_k, rows, weights, (uint8_t*)out);           \
  else                                                                                                             \
    k_moe_combine<DT, false><<<(unsigned)blocks, kThreads, 0, st>>>((const uint8_t*)y, tokens, hidden, chunks,     \
                                                                    top_k, rows, weights, (uint8_t*)out)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* grad_out, const void* y, int dt, int64_t tokens, int64_t hidden,
                                  int top_k, const int32_t* rows, const float* weights, void* grad_y,
                                  float* grad_weights, hipStream_t st) {
  const int chunks = (int)((hidden + 7) / 8);
  if (tokens > 0x7FFFFFFF) return hipErrorInvalidValue;
#define CALL(DT)                                                                                               \
  k_moe_combine_bwd<DT><<<(unsigned)tokens, kThreads, 0, st>>>((const uint8_t*)grad_out, (const uint8_t*)y,    \
                                                               tokens, hidden, chunks, top_k, rows, weights,   \
                                                               (uint8_t*)grad_y, grad_weights)
  MXQ_BY_DTYPE(dt, CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace mxq
