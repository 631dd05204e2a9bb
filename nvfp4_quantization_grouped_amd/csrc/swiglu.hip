// The experts' activation h = silu(gate) * up between the two grouped
// products, and its gradient from an input that was kept in 8 bits.
//
// All of it is one HBM stream each way, read and written past the caches except
// for what is kept, which the backward reads.  bf16 [65536, 2 * 2048], 1.08 GB
// each way: forward 185 us (5.9 TB/s), gradient 171 (6.3 TB/s), the two one after
// the other 334; with the kept codes past the caches too 176, 171 and 349, with
// every store through them the two take 375.  Without a checkpoint the forward
// takes 130-133 us (0.81 GB, 6.2 TB/s).  A lane owns 8 consecutive columns of
// gate and the same 8 of up, four lanes a block of 32 columns of each, whose
// largest magnitudes meet by DPP; inter is a multiple of 32, so no block
// straddles gate and up and every group of four lanes is whole.
//
// Keeping gate and up as E4M3 under a power of two per 32 columns (the form
// that quantize_cache_packed gives for fp8 and block_size 32) holds 1.03 bytes
// an element between forward and backward instead of 2 or 4.  The backward
// uses the kept values throughout, so it is the gradient of silu(gate) * up at
// a point within half an E4M3 step (2^-4 relative, or 2^-10 of the block's
// power of two) of the true one.
#include "moe_launch.hpp"
#include "moe_device.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t rows_that_count(const int32_t* total, int64_t rows) {
  return total ? min(rows, max((int64_t)0, (int64_t)*total)) : rows;
}

// Chunk i of this workgroup's run that starts at chunk `base` of rows x chunks:
// its row and its place in the row, by one division of 32 bits a lane.
struct Spot {
  int64_t row;
  int chunk;
};
__device__ __forceinline__ Spot spot_of(int64_t row0, unsigned first, unsigned i, unsigned chunks) {
  const unsigned at = first + i, d = at / chunks;
  return {row0 + d, (int)(at - d * chunks)};
}

// silu(gate) * up of eight columns in fp32, before its rounding to DT.  The
// compiler may fold the last product and the rounding to fp16 into one
// instruction that rounds once, and does it in some places and not in others:
// kept apart, so that every caller gets the same bits.
template <int DT>
__device__ __forceinline__ void silu_mul(const float (&g)[8], const float (&u)[8], float (&o)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o[k] = g[k] * sigmoid_f32(g[k]) * u[k];
    if constexpr (DT == DT_F16) asm("" : "+v"(o[k]));
  }
}

template <int DT, bool KEEP>
__global__ void __launch_bounds__(kThreads) k_swiglu_fwd(const uint8_t* __restrict__ gate_up, int64_t rows, int chunks,
                                                         const int32_t* __restrict__ total, uint8_t* __restrict__ h,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t count = rows_that_count(total, rows), n = rows * chunks;
  for (int64_t base = (int64_t)blockIdx.x * kThreads; base < n; base += (int64_t)gridDim.x * kThreads) {
    const int64_t row0 = base / chunks, i = base + threadIdx.x;
    if (i >= n) break;
    const Spot spot = spot_of(row0, (unsigned)(base - row0 * chunks), threadIdx.x, chunks);
    const int64_t row = spot.row;
    const int c = spot.chunk;
    if (row >= count) {
      store8<DT, true>(h, i * 8, 8, zero8<DT>());
      continue;
    }
    const int64_t at = row * 2 * chunks + c;     // chunk of gate; up is `chunks` further
    float g[8], u[8], o[8];
    to_f32<DT>(load8<DT, true>(gate_up, at * 8, 8), g);
    to_f32<DT>(load8<DT, true>(gate_up, (at + chunks) * 8, 8), u);
    silu_mul<DT>(g, u, o);
    store8<DT, true>(h, i * 8, 8, from_f32<DT>(o));
    if constexpr (KEEP) {
      const int kg = ceil_rule_exponent<FMT_FP8>(group_max_u32<4>(amax_bits(g)));
      const int ku = ceil_rule_exponent<FMT_FP8>(group_max_u32<4>(amax_bits(u)));
      store_8<false>(codes + at * 8, encode_fp8(g, pow2f(kg)));
      store_8<false>(codes + (at + chunks) * 8, encode_fp8(u, pow2f(ku)));
      if ((chunks & 15) == 0) {        // 16 lanes hold four blocks: one store of four bytes
        const uint32_t bg = scale_bytes(kg, c), bu = scale_bytes(ku, c);
        if ((c & 15) == 0) {
          store4<false>(scales + (at >> 2), bg);
          store4<false>(scales + ((at + chunks) >> 2), bu);
        }
      } else if ((c & 3) == 0) {
        scales[at >> 2] = (uint8_t)(kg + 127);
        scales[(at + chunks) >> 2] = (uint8_t)(ku + 127);
      }
    }
  }
}

// h quantized on its way out: rounded to DT, then as a block of 32 columns by
// four lanes.  bf16 [131072, 2 * 2048] to fp8, 1.35 GB: 265 us (5.1 TB/s, its
// vector instructions alone some 190), where writing h takes 267 and quantizing
// it from there 127 more.
template <int DT, bool FP4>
__global__ void __launch_bounds__(kThreads) k_swiglu_quantized(const uint8_t* __restrict__ gate_up, int64_t rows,
                                                               int chunks, const int32_t* __restrict__ total,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  const int64_t count = rows_that_count(total, rows), n = rows * chunks;
  for (int64_t base = (int64_t)blockIdx.x * kThreads; base < n; base += (int64_t)gridDim.x * kThreads) {
    const int64_t row0 = base / chunks, i = base + threadIdx.x;
    if (i >= n) break;
    const Spot spot = spot_of(row0, (unsigned)(base - row0 * chunks), threadIdx.x, chunks);
    const int c = spot.chunk;
    float o[8] = {};
    if (spot.row < count) {
      const int64_t at = spot.row * 2 * chunks + c;
      float g[8], u[8];
      to_f32<DT>(load8<DT, true>(gate_up, at * 8, 8), g);
      to_f32<DT>(load8<DT, true>(gate_up, (at + chunks) * 8, 8), u);
      silu_mul<DT>(g, u, o);
      to_f32<DT>(from_f32<DT>(o), o);
    }
    const uint32_t amax = group_max_u32<4>(amax_bits(o));
    const int k = FP4 ? floor_rule_exponent(amax) : ceil_rule_exponent<FMT_FP8>(amax);
    if constexpr (FP4) store4<true>(codes + i * 4, encode_fp4(o, pow2f(k)));
    else store_8<true>(codes + i * 8, encode_fp8(o, pow2f(k)));
    if ((chunks & 15) == 0) {
      const uint32_t b = scale_bytes(k, c);
      if ((c & 15) == 0) store4<false>(scales + (i >> 2), b);
    } else if ((c & 3) == 0) {
      scales[i >> 2] = (uint8_t)(k + 127);
    }
  }
}

template <int DT, bool KEPT>
__global__ void __launch_bounds__(kThreads) k_swiglu_bwd(const uint8_t* __restrict__ grad_h,
                                                         const uint8_t* __restrict__ gate_up,
                                                         const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t rows, int chunks,
                                                         const int32_t* __restrict__ total,
                                                         uint8_t* __restrict__ grad) {
  const int64_t count = rows_that_count(total, rows), n = rows * chunks;
  for (int64_t base = (int64_t)blockIdx.x * kThreads; base < n; base += (int64_t)gridDim.x * kThreads) {
    const int64_t row0 = base / chunks, i = base + threadIdx.x;
    if (i >= n) break;
    const Spot spot = spot_of(row0, (unsigned)(base - row0 * chunks), threadIdx.x, chunks);
    const int64_t row = spot.row;
    const int c = spot.chunk;
    const int64_t at = row * 2 * chunks + c;
    if (row >= count) {
      store8<DT, true>(grad, at * 8, 8, zero8<DT>());
      store8<DT, true>(grad, (at + chunks) * 8, 8, zero8<DT>());
      continue;
    }
    float g[8], u[8], d[8];
    to_f32<DT>(load8<DT, true>(grad_h, i * 8, 8), d);
    if constexpr (KEPT) {
      decode_fp8(*reinterpret_cast<const u32x2_any*>(codes + at * 8), e8m0_to_f32(scales[at >> 2]), g);
      decode_fp8(*reinterpret_cast<const u32x2_any*>(codes + (at + chunks) * 8),
                 e8m0_to_f32(scales[(at + chunks) >> 2]), u);
    } else {
      to_f32<DT>(load8<DT, true>(gate_up, at * 8, 8), g);
      to_f32<DT>(load8<DT, true>(gate_up, (at + chunks) * 8, 8), u);
    }
    float dg[8], du[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = sigmoid_f32(g[k]);
      // grad_h last: the factors before it are no larger than gate or up, so that a far gate's s = 0 meets no overflow
      dg[k] = d[k] * (u[k] * (s * (1.0f + g[k] * (1.0f - s))));
      du[k] = d[k] * (g[k] * s);
    }
    store8<DT, true>(grad, at * 8, 8, from_f32<DT>(dg));
    store8<DT, true>(grad, (at + chunks) * 8, 8, from_f32<DT>(du));
  }
}

unsigned grid_of(int64_t n) { return (unsigned)min((n + kThreads - 1) / kThreads, (int64_t)1 << 20); }

}  // namespace

hipError_t launch_swiglu_fwd(const void* gate_up, int dt, int64_t rows, int64_t inter, const int32_t* total, void* h,
                             uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int chunks = (int)(inter / 8);
  const unsigned grid = grid_of(rows * chunks);
#define CALL(DT)                                                                                                   \
  if (codes)                                                                                                       \
    k_swiglu_fwd<DT, true><<<grid, kThreads, 0, st>>>((const uint8_t*)gate_up, rows, chunks, total, (uint8_t*)h,   \
                                                      codes, scales);                                              \
  else                                                                                                             \
    k_swiglu_fwd<DT, false><<<grid, kThreads, 0, st>>>((const uint8_t*)gate_up, rows, chunks, total, (uint8_t*)h,  \
                                                       codes, scales)
  if (dt == DT_F32) { CALL(DT_F32); }
  else if (dt == DT_BF16) { CALL(DT_BF16); }
  else { CALL(DT_F16); }
#undef CALL
  return hipGetLastError();
}

hipError_t launch_swiglu_quantized(const void* gate_up, int dt, int64_t rows, int64_t inter, const int32_t* total,
                                   int fmt, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int chunks = (int)(inter / 8);
  const unsigned grid = grid_of(rows * chunks);
#define CALL(DT)                                                                                                   \
  if (fmt == FMT_MXFP4)                                                                                            \
    k_swiglu_quantized<DT, true><<<grid, kThreads, 0, st>>>((const uint8_t*)gate_up, rows, chunks, total, codes,   \
                                                            scales);                                               \
  else                                                                                                             \
    k_swiglu_quantized<DT, false><<<grid, kThreads, 0, st>>>((const uint8_t*)gate_up, rows, chunks, total, codes,  \
                                                             scales)
  if (dt == DT_F32) { CALL(DT_F32); }
  else if (dt == DT_BF16) { CALL(DT_BF16); }
  else { CALL(DT_F16); }
#undef CALL
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const void* grad_h, const void* gate_up, const uint8_t* codes, const uint8_t* scales,
                             int dt, int64_t rows, int64_t inter, const int32_t* total, void* grad_gate_up,
                             hipStream_t st) {
  const int chunks = (int)(inter / 8);
  const unsigned grid = grid_of(rows * chunks);
#define CALL(DT)                                                                                                      \
  if (codes)                                                                                                          \
    k_swiglu_bwd<DT, true><<<grid, kThreads, 0, st>>>((const uint8_t*)grad_h, (const uint8_t*)gate_up, codes, scales, \
                                                      rows, chunks, total, (uint8_t*)grad_gate_up);                   \
  else                                                                                                                \
    k_swiglu_bwd<DT, false><<<grid, kThreads, 0, st>>>((const uint8_t*)grad_h, (const uint8_t*)gate_up, codes,        \
                                                       scales, rows, chunks, total, (uint8_t*)grad_gate_up)
  if (dt == DT_F32) { CALL(DT_F32); }
  else if (dt == DT_BF16) { CALL(DT_BF16); }
  else { CALL(DT_F16); }
#undef CALL
  return hipGetLastError();
}

}  // namespace mxq
