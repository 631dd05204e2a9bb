// Device-side building blocks of the routed-expert layer's kernels: eight
// consecutive elements of a row as fp32 values, whatever the type.
//
// Rows have no alignment of their own (a hidden size need not be a multiple
// of anything), so the vector types below are declared with an alignment of
// one byte: gfx950's global memory instructions take such addresses, and a
// 16-byte access of an aligned row is the same instruction.
#pragma once

#include "mxq_device.hpp"

namespace mxq {

typedef u32x4_t u32x4_any __attribute__((aligned(1)));
typedef u32x2_t u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

template <int DT>
constexpr int kElemBytes = DT == DT_F32 ? 4 : 2;

// Raw bits of eight elements (4 words, 8 for fp32).
template <int DT>
struct Raw8 {
  static constexpr int kWords = DT == DT_F32 ? 8 : 4;
  uint32_t w[kWords];
};

template <int DT>
__device__ __forceinline__ float elem_value(uint32_t bits) {
  if constexpr (DT == DT_F32) return as_f32(bits);
  else if constexpr (DT == DT_BF16) return as_f32(bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
}
// fp32 -> bits of DT, nearest-even.
template <int DT>
__device__ __forceinline__ uint32_t elem_bits(float v) {
  if constexpr (DT == DT_F32) return as_u32(v);
  else if constexpr (DT == DT_BF16) return __builtin_bit_cast(unsigned short, (__bf16)v);
  else return __builtin_bit_cast(unsigned short, (_Float16)v);
}
template <int DT>
__device__ __forceinline__ uint32_t load_bits(const uint8_t* p) {
  if constexpr (DT == DT_F32) return *reinterpret_cast<const u32_any*>(p);
  else return *reinterpret_cast<const u16_any*>(p);
}
template <int DT>
__device__ __forceinline__ void store_bits(uint8_t* p, uint32_t b) {
  if constexpr (DT == DT_F32) *reinterpret_cast<u32_any*>(p) = b;
  else *reinterpret_cast<u16_any*>(p) = (uint16_t)b;
}

// 16 bytes at any address; STREAM goes past the caches (non-temporal).
template <bool STREAM>
__device__ __forceinline__ u32x4_t load16(const uint8_t* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  else return *reinterpret_cast<const u32x4_any*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint8_t* p, u32x4_t v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  else *reinterpret_cast<u32x4_any*>(p) = v;
}

template <bool STREAM>
__device__ __forceinline__ void store_8(uint8_t* p, u32x2_t v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(p));
  else *reinterpret_cast<u32x2_any*>(p) = v;
}
template <bool STREAM>
__device__ __forceinline__ void store4(uint8_t* p, uint32_t v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32_any*>(p));
  else *reinterpret_cast<u32_any*>(p) = v;
}

// Elements e .. e + 7 of the row at `row`, of which `n` (1..8) exist; the others read as 0.
template <int DT, bool STREAM = false>
__device__ __forceinline__ Raw8<DT> load8(const uint8_t* row, int64_t e, int n) {
  Raw8<DT> r;
  const uint8_t* p = row + e * kElemBytes<DT>;
  if (n == 8) {
    const u32x4_t a = load16<STREAM>(p);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    if constexpr (DT == DT_F32) {
      const u32x4_t b = load16<STREAM>(p + 16);
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < Raw8<DT>::kWords; ++i) r.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        const uint32_t b = load_bits<DT>(p + i * kElemBytes<DT>);
        if constexpr (DT == DT_F32) r.w[i] = b;
        else r.w[i / 2] |= b << (16 * (i & 1));
      }
  }
  return r;
}
template <int DT, bool STREAM = false>
__device__ __forceinline__ void store8(uint8_t* row, int64_t e, int n, const Raw8<DT>& r) {
  uint8_t* p = row + e * kElemBytes<DT>;
  if (n == 8) {
    store16<STREAM>(p, u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]});
    if constexpr (DT == DT_F32) store16<STREAM>(p + 16, u32x4_t{r.w[4], r.w[5], r.w[6], r.w[7]});
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        if constexpr (DT == DT_F32) store_bits<DT>(p + i * 4, r.w[i]);
        else store_bits<DT>(p + i * 2, (r.w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
      }
  }
}

template <int DT>
__device__ __forceinline__ void to_f32(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == DT_F32) v[i] = as_f32(r.w[i]);
    else if constexpr (DT == DT_BF16) v[i] = i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
    else v[i] = i & 1 ? f16_hi(r.w[i / 2]) : f16_lo(r.w[i / 2]);
  }
}
template <int DT>
__device__ __forceinline__ Raw8<DT> from_f32(const float (&v)[8]) {
  Raw8<DT> r;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = as_u32(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = elem_bits<DT>(v[2 * i]) | (elem_bits<DT>(v[2 * i + 1]) << 16);
  }
  return r;
}
template <int DT>
__device__ __forceinline__ Raw8<DT> zero8() {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < Raw8<DT>::kWords; ++i) r.w[i] = 0u;
  return r;
}
// Elements 0 .. n - 1 (n < 8) become 0.
template <int DT>
__device__ __forceinline__ void clear_first(Raw8<DT>& r, int n) {
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) {
      if constexpr (DT == DT_F32) r.w[i] = 0u;
      else r.w[i / 2] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
}

// fp32 bits of the largest magnitude of eight values.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, as_u32(v[i]) & 0x7FFFFFFFu);
  return m;
}
// Eight values / s as E4M3 codes, nearest-even, sign kept.
__device__ __forceinline__ u32x2_t encode_fp8(const float (&v)[8], float s) {
  return u32x2_t{enc_fp8_f2<true>(enc_fp8_f2<false>(0u, v[0], v[1], s), v[2], v[3], s),
                 enc_fp8_f2<true>(enc_fp8_f2<false>(0u, v[4], v[5], s), v[6], v[7], s)};
}
__device__ __forceinline__ void decode_fp8(u32x2_t c, float s, float (&v)[8]) {
  const f32x2_t a = dec_fp8_f2<false>(c.x, s), b = dec_fp8_f2<true>(c.x, s);
  const f32x2_t d = dec_fp8_f2<false>(c.y, s), e = dec_fp8_f2<true>(c.y, s);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = d.x; v[5] = d.y; v[6] = e.x; v[7] = e.y;
}
// Eight values / s as e2m1 codes, element 0 in the low nibble; -0.0 encodes as +0.
__device__ __forceinline__ uint32_t encode_fp4(const float (&v)[8], float s) {
  uint32_t c = enc_fp4_f2<0>(0u, v[0] + 0.0f, v[1] + 0.0f, s);
  c = enc_fp4_f2<1>(c, v[2] + 0.0f, v[3] + 0.0f, s);
  c = enc_fp4_f2<2>(c, v[4] + 0.0f, v[5] + 0.0f, s);
  return enc_fp4_f2<3>(c, v[6] + 0.0f, v[7] + 0.0f, s);
}

// E8M0 bytes of four blocks of 32 columns, block b in byte b, in every lane of
// the 16 (aligned) that hold them; k is the block's exponent, the same in its
// four lanes, whose chunks are 16 consecutive ones from a multiple of 16.
__device__ __forceinline__ uint32_t scale_bytes(int k, int chunk) {
  uint32_t b = (uint32_t)(k + 127) << (8 * ((chunk >> 2) & 3));
  b |= dpp<0x141>(b);                  // row_half_mirror: the other block of 8 lanes
  return b | dpp<0x140>(b);            // row_mirror: the other 8 lanes
}

// exp(-a) for a >= 0 to a few ulp: the rounding error of a * log2(e), and the
// part of log2(e) that fp32 drops, go back in as a factor 1 + lo ln 2 (the
// bare product loses |a| / 10 ulp).  Past a = 200 the result is 0 either way.
__device__ __forceinline__ float exp_neg(float a) {
  a = fminf(a, 200.0f);
  const float t = -a * 0x1.715476p+0f;
  const float lo = __builtin_fmaf(-a, 0x1.715476p+0f, -t) - a * 0x1.4ae0c0p-26f;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * 0x1.62e430p-1f, lo, e);
}
// 1 / (1 + exp(-x)), without overflow on either side.
__device__ __forceinline__ float sigmoid_f32(float x) {
  const float a = exp_neg(fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + a);
  return x >= 0.0f ? r : a * r;
}

// Orders LDS accesses of one wave's lanes among each other.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace mxq
