// cache_attention: attention of new tokens over the packed, paged cache.  The
// kernels; csrc/cache_attention_<format>_<type>.hip instantiate them.
//
// Mathematics.  Rows are the (token, head) pairs of one sequence that share a kv
// head, 16 to a tile and MT tiles to a wave.  A wave takes 32 positions at a
// time, transposed so that nothing changes lanes between the products:
//   S^T [32 positions, rows] = K Q^T          (16x16x32 bf16 MFMA, K decoded in registers)
//   P^T = exp2(S^T * scale * log2(e) - m)
//   O^T [channels, rows]   += V^T P^T
// A lane holds four positions of one row of each 16 x 16 tile of S^T, which are
// exactly the k slots that it feeds as P^T; the order of positions within the
// sum is free, so V^T takes the same.  The order of channels within K Q^T is
// free too: a lane's 8 channels of a step are chosen so that a lane loads 16
// consecutive bytes.  V is decoded two channels at a time for 8 positions and
// turned by v_perm.  Up to 16 or 32 rows (Attention) keys, values and
// probabilities stay in registers; LDS holds the waves' sums in the end, q where
// its parts are too many for the registers, and the marks of values that are not
// finite.  Beyond (SharedAttention) keys and values pass through LDS, decoded.
//
// Softmax.  m is a row's running maximum in units of log2, moved only when a
// score exceeds it by 2^8 (probabilities stay below 2^8 relative to it, which
// fp32 and bf16 hold as well as 1), so that most tiles neither exchange maxima
// nor rescale sums.  Sums are fp32.
//
// Roundings.  Codes times scales have at most 6 significant bits and are exact
// in bf16.  q of fp16 / fp32 enters as 2 / 3 bf16 parts (exact but for what
// lies 2^-24 below), fp16 as it is where the keys are exact in fp16 too (64
// contexts of 16384, [1, 64 / 1, 512], 237 us against 270).  Probabilities are a
// choice: one bf16 part, up to 2^-8 of each, would make the error of bf16 outputs
// 1.4 times what rounding them costs; two parts (three for fp32 outputs) leave
// nothing to see, at as many products.
// For bf16 outputs one fp16 part does (2^-11; the error is 1.01 times the
// rounding's) where the values fit fp16 exactly, which the scales tell: always
// for nvfp4, else (and where there are many rows) for scales of 2^-15 to 2^7
// (fp8) or 2^-23 to 2^13 (mxfp4).  A workgroup that meets others starts its piece
// again with two bf16 parts: blocks of zeros are among them, as they are
// quantized with byte 1 (64-token trees with a row of zeros in every page 300 us
// against 259).
//
// What bounds it.  One token a sequence: memory (64 contexts of up to 16384, 8
// heads of 8 queries, mxfp4: 638 MB in 138 us, 4.6 TB/s).  Trees: the products
// and what feeds them (64 tokens, 8 contexts of up to 16384, fp8: 167 GFLOP in
// 252 us, 660 TFLOP/s; when it took 325, 137 without its products and 275
// without its loads).  Short calls: beginning and ending a piece, 12 to 15 us of
// waits that follow one another (lengths and shares 2.4, queries 4.5, first rows
// 2.3, first products 2.5, sums written 2 to 4 us).
#pragma once

#include <type_traits>
#include <utility>

#include "cache_device.hpp"

namespace mxq {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

constexpr int kAttnThreads = 256;
constexpr int kTile = 32;                    // positions of a wave's tile
// Log2 units by which probabilities may exceed 1, and (fp16) what the largest is when the maximum moves: fp16's range is
// then 2^-30 to 2^14 times the row's largest, so that n small ones lose at most n 2^-31 of the sum.
template <bool HALF>
constexpr float kOver = HALF ? 14.0f : 8.0f;
template <bool HALF>
constexpr float kAtMove = HALF ? 6.0f : 0.0f;

struct AttnDims {
  int sequences, tokens, heads, group, kv_heads, width, page_shift;
  int row_tiles;        // tiles of a kernel's rows of a sequence and kv head, all tokens counted
  int workgroups;       // that share the steps (split), or 0: one workgroup for each problem
  bool mask_each;
  int64_t pages;
  float scale;          // its size, times log2(e), no less than 2^-149: -inf times it is -inf
  bool negative;        // its sign, which q takes
};
struct AttnArgs {
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t *table, *lengths, *counts;
  const uint8_t *q, *mask;
  uint8_t* out;
  float* lse;
  float* parts;         // two slots for each workgroup: sums [rows][D], then m and l [rows]
  int block_shift;
  AttnDims d;
};

// ------------------------------------------------------------------- shapes
// Whether keys and q multiply as fp16: q is, and the keys fit whatever their scales are.
template <int DT, int FMT>
constexpr bool kHalfKeys = DT == DT_F16 && FMT == FMT_NVFP4;
template <int DT, int FMT>
constexpr int kQParts = DT == DT_BF16 || kHalfKeys<DT, FMT> ? 1 : DT == DT_F16 ? 2 : 3;
template <int DT>
constexpr int kPParts = DT == DT_F32 ? 3 : 2;

// Whether fp16 probabilities serve whatever the scales are.  The other formats take them first where there are many rows
// (products bound those calls: 64-token trees 311 us, with them 273); where a wave's loads do, the second way's registers
// cost more than the products save.
template <int DT, int FMT>
constexpr bool kHalfOnly = DT == DT_BF16 && FMT == FMT_NVFP4;

template <int FMT, int D>
struct Shape {
  static constexpr bool kFp8 = FMT == FMT_FP8;
  static constexpr int kRowBytes = kFp8 ? D : D / 2;
  // K: a lane takes KC channels of a unit; four lanes' channels are neighbours
  static constexpr int KC = kFp8 ? 16 : (D >= 128 ? 32 : 16);
  static constexpr int KU = D / (4 * KC);                   // units of a row
  static constexpr int KW = kFp8 ? KC / 4 : KC / 8;         // words of a unit
  static constexpr int KS = KC / 16;                        // scale bytes of a unit
  static constexpr int kHalves = KC / 8;                    // MFMA steps of a unit
  static constexpr int kSteps = D / 32;
  // V: a lane takes VC channels of a unit; 16 lanes' channels are neighbours
  static constexpr int VC = D / 16 > 16 && kFp8 ? 16 : D / 16;
  static constexpr int VU = D / 16 / VC;
  static constexpr int VB = kFp8 ? VC : VC / 2;             // bytes of a unit
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int VS = VC > 16 ? 2 : 1;                // scale bytes of a unit
};

template <int N, class F, int... I>
__device__ __forceinline__ void static_for_(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_<N>(f, std::make_integer_sequence<int, N>{});
}

// Channels 2 I and 2 I + 1 of a unit's words as a pair of bf16.
template <int FMT, int I>
__device__ __forceinline__ uint32_t decode_pair(const uint32_t* w, float s) {
  if constexpr (FMT == FMT_FP8) return dec_fp8_bf16x2<(I & 1) != 0>(w[I / 2], s);
  else return dec_fp4_bf16x2<I & 3>(w[I / 4], s);
}
// The same as a pair of fp16.
template <int FMT, int I>
__device__ __forceinline__ uint32_t decode_pair_half(const uint32_t* w, float s) {
  if constexpr (FMT == FMT_FP8)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[I / 2], s, (I & 1) != 0));
  else return dec_fp4_f16x2<I & 3>(w[I / 4], s);
}
template <bool HALF, int FMT, int I>
__device__ __forceinline__ uint32_t decode_value(const uint32_t* w, float s) {
  if constexpr (HALF) return decode_pair_half<FMT, I>(w, s);
  else return decode_pair<FMT, I>(w, s);
}
// Scale byte -> scale for the conversions, which take its exponent: for E8M0 that is the byte (0 means 2^-127 and 0xFF NaN
// there too, bit for bit over every code).
template <int FMT>
__device__ __forceinline__ float scale_operand(uint32_t b) {
  if constexpr (FMT == FMT_NVFP4) return scale_value<FMT>(b);
  else return as_f32(b << 23);
}
// Whether a scale is more than its exponent (an E4M3 byte that is not what quantize_cache_packed writes): mantissa bits
// (NaN has some), a sign, or 0.
__device__ __forceinline__ bool beyond_exponent(float s) { return (as_u32(s) & 0x807FFFFFu) != 0 || s == 0.0f; }
// Such a scale, 2^e (1 + b1 / 2 + b2 / 4 + b3 / 8), in four passes that each take a power of two: 2^e, then 2^(e - pass)
// where that bit is set, and next to nothing (2^-127) where it is not.  NaN stays NaN in the first.
__device__ __forceinline__ float scale_in_pass(float s, int pass) {
  const uint32_t u = as_u32(s), e = u >> 23 & 0xFFu;
  if (pass == 0) return e == 255u ? s : as_f32(e << 23);
  return e != 255u && (u >> (23 - pass) & 1u) ? as_f32((e - pass) << 23) : 0.0f;
}

// The least code (by size) that is not finite in bf16 under a scale byte; one past the largest where all are.
template <int FMT>
__device__ __forceinline__ int least_odd(int e) {
  if constexpr (FMT == FMT_NVFP4) return (e & 0x7F) == 0x7F ? 0 : 8;
  else if constexpr (FMT == FMT_FP8) return e == 255 ? 0 : min(127, max(262 - e, 0) << 3);   // code 0x7F is NaN itself
  else return e == 255 ? 0 : min(8, max(256 - e, 0) << 1);
}

// The same of a word's codes: the top bit of each that is +inf or NaN, and of each that is -inf or NaN.  `least` is least_odd
// of their scale byte, `more` kHalf - least in each code.
template <int FMT>
struct Odd {
  static constexpr uint32_t kOnes = FMT == FMT_FP8 ? 0x01010101u : 0x11111111u, kTop = FMT == FMT_FP8 ? 0x80808080u : 0x88888888u;
  static constexpr int kBits = FMT == FMT_FP8 ? 8 : 4, kHalf = 1 << (kBits - 1);
  uint32_t sign[2];
  __device__ __forceinline__ Odd(uint32_t word, uint32_t more, bool nan_scale) {
    const uint32_t f = ((word & ~kTop) + more) & kTop;
    const uint32_t nan = nan_scale ? kTop : FMT == FMT_FP8 ? ((word & ~kTop) + kOnes) & kTop : 0u;   // (0x7F is NaN)
    sign[0] = f & (~word | nan);
    sign[1] = f & (word | nan);
  }
  __device__ __forceinline__ uint32_t any() const { return sign[0] | sign[1]; }
  // All bits of those codes.
  __device__ __forceinline__ uint32_t codes() const { return (any() >> (kBits - 1)) * (2 * kHalf - 1); }
};
// Scale bytes from here on make some finite code infinite in bf16 (nvfp4's never do).
template <int FMT>
constexpr uint32_t kPastBf16 = FMT == FMT_FP8 ? 247 : 253;

// What infinite values make of an output: marks 1 for +inf, 2 for -inf, 3 for both (or NaN).
__device__ __forceinline__ float marked_value(float x, uint32_t marks) {
  const float inf = __builtin_inff();
  return marks == 0 ? x : marks == 1 ? inf : marks == 2 ? -inf : __builtin_nanf("");
}
// What a part's sums are multiplied by whose maximum is m, where the whole's is `top`.  Never 0, so that an infinity stays
// one however small the part's share is: 2^-149 in the place of a share below 2^-126, as others' sums, of n values of up to
// 2^8 |v|, come to nothing by it (n 2^-141 of the largest value).  A part that met nothing, or NaN alone, has an m of -inf
// and an l of 0 or NaN.
__device__ __forceinline__ float share_of_part(float m, float l, float top) {
  return m == -__builtin_inff() ? l : fmaxf(__builtin_amdgcn_exp2f(m - top), 0x1p-149f);
}

__device__ __forceinline__ bf16x8_t as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{a, b, c, d});
}
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
// Values times probabilities, bf16 or fp16.
template <bool HALF>
__device__ __forceinline__ f32x4_t mfma_value(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
// Whether E8M0 scale bytes keep every code of theirs exact in fp16: 448 or 6 times the scale within 65504, 2^-9 or 0.5
// times it no less than 2^-24.
template <int FMT>
__device__ __forceinline__ bool fits_half(uint32_t least, uint32_t most) {
  if constexpr (FMT == FMT_FP8) return least >= 112 && most <= 134;
  else return least >= 104 && most <= 140;
}
template <bool HALF>
__device__ __forceinline__ f32x4_t mfma_key(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return mfma_value<HALF>(__builtin_bit_cast(u32x4_t, a), __builtin_bit_cast(u32x4_t, b), c);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));     // one conversion of two
}
// (-1, 0) and (0, -1) in bf16.  Held in registers: the compiler makes 32-bit float constants of such literals, which a
// dot product then misreads.
struct MinusOne {
  uint32_t lo = 0x0000BF80u, hi = 0xBF800000u;
  __device__ __forceinline__ MinusOne() { asm("" : "+s"(lo), "+s"(hi)); }
};
// The next bf16 part of eight values, which keep what is left: exact, and one instruction a value as a dot product of a
// pair.  (A NaN or an infinity takes its neighbour with it: both are of one row, whose sum is NaN.)
__device__ __forceinline__ bf16x8_t take_part(float (&x)[8], bool last, const MinusOne& minus) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    if (!last) {
      const bf16x2_t part = __builtin_bit_cast(bf16x2_t, w[i]);
      x[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(part, __builtin_bit_cast(bf16x2_t, minus.lo), x[2 * i], false);
      x[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(part, __builtin_bit_cast(bf16x2_t, minus.hi), x[2 * i + 1], false);
    }
  }
  return as_bf16x8(w[0], w[1], w[2], w[3]);
}
// q's parts: eight values of them.
template <int DT, int FMT>
__device__ __forceinline__ void parts_of(float (&x)[8], const MinusOne& minus, bf16x8_t (&part)[kQParts<DT, FMT>]) {
  if constexpr (kHalfKeys<DT, FMT>) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{x[2 * i], x[2 * i + 1]}, f16x2_t));
    part[0] = __builtin_bit_cast(bf16x8_t, w);
  } else {
#pragma unroll
    for (int p = 0; p < kQParts<DT, FMT>; ++p) part[p] = take_part(x, p == kQParts<DT, FMT> - 1, minus);
  }
}
// A loaded value, not looked at before this point: what is computed from it (a scale from its byte) would otherwise be
// moved up to the load, and the wait for the load with it, before the products that are to hide it.
template <int N>
__device__ __forceinline__ void from_here(uint32_t (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}
template <int N, int M>
__device__ __forceinline__ void from_here(uint32_t (&x)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i) from_here(x[i]);
}
template <int N, int M, int L>
__device__ __forceinline__ void from_here(uint32_t (&x)[N][M][L]) {
#pragma unroll
  for (int i = 0; i < N; ++i) from_here(x[i]);
}
// The first of eight moved behind the others: what a loop does to the first of them it does to each, once in its code.
__device__ __forceinline__ void to_the_end(uint32_t (&x)[8]) {
  const uint32_t first = x[0];
#pragma unroll
  for (int i = 0; i < 7; ++i) x[i] = x[i + 1];
  x[7] = first;
}
template <int N>
__device__ __forceinline__ void to_the_end(uint32_t (&x)[8][N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t first = x[0][n];
#pragma unroll
    for (int i = 0; i < 7; ++i) x[i][n] = x[i + 1][n];
    x[7][n] = first;
  }
}
template <int N, int M>
__device__ __forceinline__ void to_the_end(uint32_t (&x)[8][N][M]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint32_t first = x[0][n][m];
#pragma unroll
      for (int i = 0; i < 7; ++i) x[i][n][m] = x[i + 1][n][m];
      x[7][n][m] = first;
    }
}
// Over the four lanes that hold a row (16 apart).
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A value that every lane of a wave reads, through the scalar cache: the wait for it is not a wait for the vector loads
// before it.  Tables and lengths do not change while a kernel runs.
__device__ __forceinline__ int uniform_load(const int32_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  return ((Scalar)(uintptr_t)p)[i];
}

// --------------------------------------------------------------- the schedule
// A problem is a sequence, a kv head and a tile of A::kRows rows; its work is its steps of A::kStep positions.
struct Work {
  int known, end, count;     // cached positions, those and the drafted ones, tokens that are no padding
  int steps, tiles;          // of each problem; row tiles that hold such a token
};
template <class A>
__device__ __forceinline__ Work work_of(const AttnArgs& a, int length, int count) {
  Work w;
  w.known = cached_positions(length, a.d.width, 1 << a.d.page_shift);
  w.count = min(max(count, 0), a.d.tokens);
  w.end = w.count > 0 ? min(w.known + w.count, a.d.width << a.d.page_shift) : 0;
  w.steps = (w.end + A::kStep - 1) / A::kStep;
  w.tiles = (w.count * a.d.group + A::kRows - 1) / A::kRows;
  return w;
}
// Of a sequence that the whole workgroup works on, in scalar registers.
template <class A>
__device__ __forceinline__ Work work_of_all(const AttnArgs& a, int b) {
  return work_of<A>(a, uniform_load(a.lengths, b), a.counts ? uniform_load(a.counts, b) : a.d.tokens);
}
// Units of a thread's sequence, all its problems together: steps, and for each problem kStart before them, as many as
// beginning and ending a piece takes the time of (12 to 18 us), so that a workgroup whose share ends one problem and begins
// another does fewer steps (16-token trees 105 -> 97 us, 100 and 98 with 2 and 6 of them; [4, 8192, 512] 47 -> 42, 64
// contexts of 16384 142 -> 138).
template <class A>
__device__ __forceinline__ int units_of(const AttnArgs& a, int b) {
  if (b >= a.d.sequences) return 0;
  const Work w = work_of<A>(a, a.lengths[b], a.counts ? a.counts[b] : a.d.tokens);
  return w.steps > 0 ? (w.steps + A::kStart) * w.tiles * a.d.kv_heads : 0;
}
// Units [first, last) of all problems' that workgroup w of g takes.
__device__ __forceinline__ int share_of(int w, int total, int g) { return (int)((int64_t)w * total / g); }
// The workgroup that takes unit u.
__device__ __forceinline__ int owner_of(int u, int total, int g) { return (int)((((int64_t)u + 1) * g - 1) / total); }

// A part of a problem that several workgroups share: sums (rows * D, in A's order), then m and l [rows].
template <class A>
constexpr int64_t kSlotFloats = (int64_t)A::kRows * (A::kDim + 2);

// Eight (or four) channels of an output row, and with the first of them its lse.
template <int DT, int N>
__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t row, int dim, int ch, const float (&sums)[N], float top,
                                          float sum) {
  float x[8] = {};
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = sum == 0.0f ? 0.0f : sums[e] / sum;
  const Raw8<DT> r = from_f32<DT>(x);
  uint8_t* at = a.out + (row * dim + ch) * kElemBytes<DT>;
  if constexpr (N == 8) store8<DT>(at, 0, 8, r);
  else if constexpr (DT == DT_F32) *reinterpret_cast<u32x4_t*>(at) = u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]};
  else *reinterpret_cast<u32x2_t*>(at) = u32x2_t{r.w[0], r.w[1]};
  if (a.lse && ch == 0)
    a.lse[row] = sum == 0.0f ? -__builtin_inff()
                 : top == -__builtin_inff() ? sum : __builtin_fmaf(top, 0x1.62e430p-1f, logf(sum));
}

// Which positions of tile t each row attends to (a bit each, in the lane's order), the scores of the others -inf.
// row0: this lane's row of the first 16.
template <int MT>
__device__ __forceinline__ void mask_scores(const AttnArgs& a, const Work& w, int b, int t, bool there0, bool there1,
                                            int row0, int quarter, f32x4_t (&s)[MT][2], uint32_t (&may)[MT]) {
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int token = (row0 + mt * 16) / a.d.group;
    const uint8_t* see = a.mask ? a.mask + ((int64_t)(a.d.mask_each ? b : 0) * a.d.tokens +
                                            min(token, a.d.tokens - 1)) * a.d.tokens : nullptr;
    may[mt] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pos = t * kTile + (i / 4) * 16 + quarter * 4 + i % 4, j = pos - w.known;
      bool ok = j <= token;
      if (see) ok = j < 0 || see[min(max(j, 0), a.d.tokens - 1)] != 0;
      ok = ok && (i < 4 ? there0 : there1) && pos < w.end && token < w.count;
      may[mt] |= (uint32_t)ok << i;
      s[mt][i / 4][i % 4] = ok ? s[mt][i / 4][i % 4] : -__builtin_inff();
    }
  }
}

// Probabilities of a tile's scores in bf16 parts, and the rows' running maximum m, sum l and sums o.
// (m is what the exponents are taken relative to; for fp16 a row's largest probability is 2^6 when it moves.)
template <bool HALF, int MT, int PP, int NT>
__device__ __forceinline__ void softmax_step(const f32x4_t (&s)[MT][2], float scale, const MinusOne& minus, float (&m)[MT],
                                             float (&l)[MT], f32x4_t (&o)[MT][NT], u32x4_t (&p)[MT][PP]) {
  float top[MT];
  bool past = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    top[mt] = s[mt][0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top[mt] = fmaxf(top[mt], s[mt][i / 4][i % 4]);
    top[mt] *= scale;
    past |= top[mt] > m[mt] + kOver<HALF>;
  }
  if (__ballot(past) != 0) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float to = fmaxf(m[mt], row_max(top[mt]) - kAtMove<HALF>);
      const float keep = m[mt] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[mt] - to);
      m[mt] = to;
      l[mt] *= keep;
#pragma unroll
      for (int c = 0; c < NT; ++c) o[mt][c] *= keep;
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float sub = m[mt] == -__builtin_inff() ? 0.0f : m[mt];
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[mt][i / 4][i % 4], scale, -sub));
      l[mt] += e[i];
    }
#pragma unroll
    for (int part = 0; part < PP; ++part) {
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[mt][part][i] =
              __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{e[2 * i], e[2 * i + 1]}, f16x2_t));
      } else {
        p[mt][part] = __builtin_bit_cast(u32x4_t, take_part(e, part == PP - 1, minus));
      }
    }
  }
}

// ------------------------------------------------------------------ one piece
template <int DT, int FMT, int D, int MT, bool HALF>
struct Attention {
  using S = Shape<FMT, D>;
  static_assert(!HALF || kHalfOnly<DT, FMT>, "a piece is not started again here");
  using Other = void;
  static constexpr int QP = kQParts<DT, FMT>, PP = HALF ? 1 : kPParts<DT>, kDim = D, kRows = 16 * MT, kStep = 4 * kTile;
  static constexpr int kTilesV = D / 16, kType = DT;
  static constexpr bool kFragments = false;                // parts are rows
  // waves of a SIMD that the registers are kept to, which is workgroups of a CU
  static constexpr int kWaves = D * MT <= 128 ? 3 : D * MT <= 256 ? 2 : 1;
  static constexpr int kThreads = kAttnThreads, kResident = kWaves, kStart = 4, kFew = 14;
  // q's fragments stay in registers up to 32 of them, else in LDS
  static constexpr bool kQInRegs = D * QP * MT <= 256;
  static constexpr int kPad = D + 4;
  static constexpr int kQBytes = kQInRegs ? 0 : QP * kRows * D * 2;
  // the four waves' sums join in as many buffers as 34 KB hold, in turns
  static constexpr int kBuffers = D * MT <= 128 ? 4 : D * MT <= 256 ? 2 : 1;
  static constexpr int kSumBytes = kBuffers * kRows * kPad * 4;
  static constexpr int kMarkBytes = kAttnThreads * S::VU * S::VW * 4;
  static constexpr int kLdsBytes = kQBytes + kMarkBytes > kSumBytes ? kQBytes + kMarkBytes : kSumBytes;

  struct Shared {
    __attribute__((aligned(16))) uint8_t big[kLdsBytes];   // q's fragments, then the waves' sums
    __attribute__((aligned(16))) uint8_t nan[kRows * D];   // marks of outputs that a value that is not finite reached
    float m[4][kRows], l[4][kRows];
    int first[kThreads];                                   // prefix sums of the schedule
    int sums[4];
  };

  const AttnArgs& a;
  Shared& sm;
  int lane, col, quarter;
  const int wave;
  const MinusOne minus;
  // the problem
  int b, kv, tile;
  Work w;

  __device__ __forceinline__ Attention(const AttnArgs& args, Shared& shared)
      : a(args), sm(shared), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
    place();
  }
  // The lane's place, anew: what is computed from it is not kept across pieces (some 25 registers of addresses).
  __device__ __forceinline__ void place() {
    lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    col = lane & 15;
    quarter = lane >> 4;
  }

  // Element offset of row r of the problem in q and out; r < tokens * group.
  __device__ __forceinline__ int64_t row_at(int r) const {
    const int i = r / a.d.group, g = r - i * a.d.group;
    return (((int64_t)b * a.d.tokens + i) * a.d.heads + kv * a.d.group + g);
  }
  __device__ __forceinline__ int row_of(int mt) const { return tile * kRows + mt * 16 + col; }

  // ----- q
  __device__ __forceinline__ void q_fragment(int mt, int step, bf16x8_t (&part)[QP]) const {
    const int u = step / S::kHalves, h = step % S::kHalves;
    const int ch = u * 4 * S::KC + quarter * S::KC + h * 8, r = row_of(mt);
    float x[8] = {};
    if (r < a.d.tokens * a.d.group) to_f32<DT>(load8<DT>(a.q, row_at(r) * D + ch, 8), x);
    if (a.d.negative)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = -x[i];
    parts_of<DT, FMT>(x, minus, part);
  }
  struct Q {
    bf16x8_t f[kQInRegs ? MT : 1][kQInRegs ? S::kSteps : 1][QP];
  };
  __device__ __forceinline__ void load_q(Q& q) const {
    if constexpr (kQInRegs) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) q_fragment(mt, s, q.f[mt][s]);
    } else {
      for (int i = wave; i < MT * S::kSteps; i += 4) {
        bf16x8_t part[QP];
        q_fragment(i / S::kSteps, i % S::kSteps, part);
#pragma unroll
        for (int p = 0; p < QP; ++p)
          *reinterpret_cast<bf16x8_t*>(sm.big + (((i * QP + p) * 64) + lane) * 16) = part[p];
      }
      __syncthreads();
    }
  }
  __device__ __forceinline__ bf16x8_t q_part(const Q& q, int mt, int step, int p) const {
    if constexpr (kQInRegs) return q.f[mt][step][p];
    else
      return *reinterpret_cast<const bf16x8_t*>(sm.big + ((((mt * S::kSteps + step) * QP + p) * 64) + lane) * 16);
  }

  // ----- rows of a tile
  struct Pages {
    int page[2];        // of the tile's halves of 16 positions; 0 where there is none
    bool there[2];
  };
  __device__ __forceinline__ Pages pages_of(int t) const {
    Pages p;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = (t * kTile + h * 16) >> a.d.page_shift;
      const int page = uniform_load(a.table, (int64_t)b * a.d.width + min(slot, a.d.width - 1));
      p.there[h] = slot < a.d.width && (uint32_t)page < (uint32_t)a.d.pages;
      p.page[h] = p.there[h] ? page : 0;
    }
    return p;
  }
  // Row in the pools of the first position of half h of tile t.
  __device__ __forceinline__ int64_t pool_row(const Pages& p, int t, int h) const {
    const int in_page = (t * kTile + h * 16) & ((1 << a.d.page_shift) - 1);
    return (((int64_t)p.page[h] * a.d.kv_heads + kv) << a.d.page_shift) + in_page;
  }
  struct K {
    uint32_t w[2][S::KU][S::KW];
    uint32_t s[2][S::KU][S::KS];
  };
  struct V {
    uint32_t w[8][S::VU][S::VW];
    uint32_t s[8][S::VU][S::VS];
  };
  __device__ __forceinline__ void load_k(K& k, const Pages& p, int t) const {
    const int blocks = D >> a.block_shift;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = pool_row(p, t, h);
      const uint8_t* codes = a.k_codes + row * S::kRowBytes;
      const uint8_t* scales = a.k_scales + row * blocks;
#pragma unroll
      for (int u = 0; u < S::KU; ++u) {
        const uint8_t* at = codes + (uint32_t)(col * S::kRowBytes + quarter * S::KW * 4) + u * S::KW * 16;
        if constexpr (S::KW == 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at);
          k.w[h][u][0] = v.x; k.w[h][u][1] = v.y; k.w[h][u][2] = v.z; k.w[h][u][3] = v.w;
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at);
          k.w[h][u][0] = v.x; k.w[h][u][1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < S::KS; ++i)
          k.s[h][u][i] = scales[(uint32_t)(col * blocks + (((u * 4 + quarter) * S::KC + i * 16) >> a.block_shift))];
      }
    }
  }
  __device__ __forceinline__ void load_v(V& v, const Pages& p, int t) const {
    const int blocks = D >> a.block_shift;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t row = pool_row(p, t, j / 4);
      const uint8_t* codes = a.v_codes + row * S::kRowBytes;
      const uint8_t* scales = a.v_scales + row * blocks;
#pragma unroll
      for (int u = 0; u < S::VU; ++u) {
        const uint8_t* at = codes + (uint32_t)(quarter * 4 * S::kRowBytes + col * S::VB) + (j % 4 * S::kRowBytes + u * 16 * S::VB);
        if constexpr (S::VB == 2) v.w[j][u][0] = *reinterpret_cast<const uint16_t*>(at);
        else if constexpr (S::VB == 4) v.w[j][u][0] = *reinterpret_cast<const uint32_t*>(at);
        else if constexpr (S::VB == 8) {
          const u32x2_t x = *reinterpret_cast<const u32x2_t*>(at);
          v.w[j][u][0] = x.x; v.w[j][u][1] = x.y;
        } else {
          const u32x4_t x = *reinterpret_cast<const u32x4_t*>(at);
          v.w[j][u][0] = x.x; v.w[j][u][1] = x.y; v.w[j][u][2] = x.z; v.w[j][u][3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < S::VS; ++i)
          v.s[j][u][i] = (scales + j % 4 * blocks)[(uint32_t)(quarter * 4 * blocks + ((u * 16 * S::VC + col * S::VC + i * 16) >> a.block_shift))];
      }
    }
  }

  // ----- products
  // Scales that are more than exponents: their sign and zero go into the codes (word by word; a unit's scales each hold
  // for as many words), and the rest takes four passes.  Returns the number of passes.
  template <int ROWS, int UNITS, int SCALES, int WORDS>
  __device__ __forceinline__ static int passes_of(uint32_t (&w)[ROWS][UNITS][WORDS], const uint32_t (&s)[ROWS][UNITS][SCALES]) {
    if constexpr (FMT != FMT_NVFP4) return 1;
    bool any = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < SCALES; ++i) any |= beyond_exponent(scale_value<FMT>(s[r][u][i]));
    if (__ballot(any) == 0) return 1;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          const float f = scale_value<FMT>(s[r][u][i * SCALES / WORDS]);
          w[r][u][i] = f == 0.0f ? 0u : w[r][u][i] ^ (as_u32(f) >> 31) * 0x88888888u;
        }
    return 4;
  }
  __device__ __forceinline__ static float scale_of(uint32_t byte, int pass, int passes) {
    const float s = scale_operand<FMT>(byte);
    if constexpr (FMT != FMT_NVFP4) return s;
    return passes == 1 ? s : scale_in_pass(s, pass);
  }
  // S^T += K Q^T.  The two halves' sums take turns, so that a product seldom waits for the one before it.
  __device__ __forceinline__ void scores(const K& k, const Q& q, int pass, int passes, f32x4_t (&s)[MT][2]) const {
    static_for<S::KU>([&](auto U) {
      constexpr int u = decltype(U)::value;
      float sc[2][S::KS];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::KS; ++i) sc[h][i] = scale_of(k.s[h][u][i], pass, passes);
      static_for<S::kHalves>([&](auto H) {
        constexpr int hf = decltype(H)::value, is = hf / 2 < S::KS ? hf / 2 : 0;
        bf16x8_t key[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4];
          static_for<4>([&](auto I) {
            x[decltype(I)::value] = decode_value<kHalfKeys<DT, FMT>, FMT, hf * 4 + decltype(I)::value>(k.w[h][u], sc[h][is]);
          });
          key[h] = as_bf16x8(x[0], x[1], x[2], x[3]);
        }
#pragma unroll
        for (int p = 0; p < QP; ++p)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const bf16x8_t f = q_part(q, mt, u * S::kHalves + hf, p);
#pragma unroll
            for (int h = 0; h < 2; ++h) s[mt][h] = mfma_key<kHalfKeys<DT, FMT>>(key[h], f, s[mt][h]);
          }
      });
    });
  }
  // O^T += V^T P^T.
  __device__ __forceinline__ void values(const V& v, const u32x4_t (&p)[MT][PP], int pass, int passes, f32x4_t (&o)[MT][kTilesV]) const {
    static_for<S::VU>([&](auto U) {
      constexpr int u = decltype(U)::value;
      float sc[8][S::VS];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < S::VS; ++i) sc[j][i] = scale_of(v.s[j][u][i], pass, passes);
      static_for<S::VC / 2>([&](auto I) {
        constexpr int i = decltype(I)::value, is = i / 8 < S::VS ? i / 8 : 0;
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = decode_value<HALF, FMT, i>(v.w[j][u], sc[j][is]);
        uint32_t y[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[0][j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
          y[1][j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
        }
        const int t = u * S::VC + 2 * i;
#pragma unroll
        for (int part = 0; part < PP; ++part)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][t + half] =
                  mfma_value<HALF>(u32x4_t{y[half][0], y[half][1], y[half][2], y[half][3]}, p[mt][part], o[mt][t + half]);
      });
    });
  }

  // Whether a value of the tile may be infinite in bf16.
  __device__ __forceinline__ static bool past_bf16(const V& v) {
    if constexpr (FMT == FMT_NVFP4) return false;
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int u = 0; u < S::VU; ++u)
#pragma unroll
        for (int i = 0; i < S::VS; ++i) most = max(most, v.s[j][u][i]);
    return __ballot(most >= kPastBf16<FMT>) != 0;
  }
  // The values of a tile that not every row attends to, or that holds infinities.  Those of rows that are no position become
  // 0.  A value that is not finite counts for the rows that attend to it alone, whatever its probability's parts are: it
  // becomes 0 here (0 times it is NaN) and is marked for those rows, whose sums are set in the end.
  __device__ __forceinline__ void clean(const Pages& now, int t, const uint32_t (&may)[MT], V& v) const {
    using Codes = Odd<FMT>;
    constexpr int kWords = S::VU * S::VW, kCodes = S::VC / S::VW;
    constexpr uint32_t kUnit = FMT == FMT_NVFP4 ? 0x38u : 127u;        // a scale of 1
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pos = t * kTile + (j / 4) * 16 + quarter * 4 + j % 4;
      const bool none = !now.there[j / 4] || pos >= w.end;
#pragma unroll
      for (int u = 0; u < S::VU; ++u) {
        uint32_t more[S::VS];
#pragma unroll
        for (int i = 0; i < S::VS; ++i) {
          v.s[j][u][i] = none ? kUnit : v.s[j][u][i];
          more[i] = (Codes::kHalf - least_odd<FMT>(v.s[j][u][i])) * Codes::kOnes;
        }
#pragma unroll
        for (int i = 0; i < S::VW; ++i) {
          v.w[j][u][i] = none ? 0u : v.w[j][u][i];
          any |= (v.w[j][u][i] & ~Codes::kTop) + more[i * S::VS / S::VW];
        }
      }
    }
    if (__ballot((any & Codes::kTop) != 0) == 0) return;
    // the marks, a position at a time (its values first in line), in a loop over its codes, whose words lie in LDS behind
    // q's fragments
    uint32_t* words = reinterpret_cast<uint32_t*>(sm.big + kQBytes) + (wave * 64 + lane) * kWords;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      uint32_t more[S::VU][S::VS];
      bool nan[S::VU][S::VS];
#pragma unroll
      for (int u = 0; u < S::VU; ++u)
#pragma unroll
        for (int i = 0; i < S::VS; ++i) {
          const int least = least_odd<FMT>(v.s[0][u][i]);
          more[u][i] = (Codes::kHalf - least) * Codes::kOnes;
          nan[u][i] = least == 0;
          v.s[0][u][i] = nan[u][i] ? kUnit : v.s[0][u][i];
        }
#pragma unroll 1
      for (int sign = 0; sign < 2; ++sign) {
#pragma unroll
        for (int u = 0; u < S::VU; ++u)
#pragma unroll
          for (int i = 0; i < S::VW; ++i) {
            const Codes f(v.w[0][u][i], more[u][i * S::VS / S::VW], nan[u][i * S::VS / S::VW]);
            words[u * S::VW + i] = sign ? f.sign[1] : f.sign[0];
          }
#pragma unroll 1
        for (int i = 0; i < kWords * kCodes; ++i) {
          const int word = i / kCodes, code = i - word * kCodes;
          const uint64_t all = __ballot(words[word] >> (code * Codes::kBits + Codes::kBits - 1) & 1u);
          // the quarter's lanes hold this channel of their units, and the rows of the same positions
          for (uint32_t lanes = (uint32_t)(all >> (quarter * 16)) & 0xFFFFu; lanes != 0; lanes &= lanes - 1) {
            const int channel = word / S::VW * 16 * S::VC + __builtin_ctz(lanes) * S::VC + word % S::VW * kCodes + code;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const int at = (mt * 16 + col) * D + channel;
              if (may[mt] >> j & 1) atomicOr(reinterpret_cast<uint32_t*>(sm.nan) + at / 4, (1u + sign) << (at % 4 * 8));
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < S::VU; ++u)
#pragma unroll
        for (int i = 0; i < S::VW; ++i)
          v.w[0][u][i] &= ~Codes(v.w[0][u][i], more[u][i * S::VS / S::VW], nan[u][i * S::VS / S::VW]).codes();
      to_the_end(v.w);
      to_the_end(v.s);
    }
  }

  // Steps [first, last) of the problem, this wave's tile of each; `whole`: they are all, else the sums go to `slot`.
  __device__ __forceinline__ bool piece(int first, int last, bool whole, float* slot) {
    place();
    for (int i = wave * 64 + lane; i < kRows * D / 16; i += kAttnThreads)
      *reinterpret_cast<u32x4_t*>(sm.nan + i * 16) = u32x4_t{0u, 0u, 0u, 0u};
    Q q;
    load_q(q);
    f32x4_t o[MT][kTilesV];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < kTilesV; ++t) o[mt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[mt] = -__builtin_inff();
      l[mt] = 0.0f;
    }
    __syncthreads();
    int t = first * 4 + wave;
    const int end = min(last * 4, (w.end + kTile - 1) / kTile);
    if (t < end) {
      Pages now = pages_of(t);
      int ahead = t + 4 < end ? t + 4 : t;
      Pages next = pages_of(ahead);
      K k;
      V v;
      load_k(k, now, t);
      load_v(v, now, t);
      // the first bytes, as words: were all of them bytes that are widened, the widening would wait at the loads
      from_here(k.s);
      from_here(v.s);
      // One tile, while the next one's rows are on their way: its keys from the scores on, its values from the values on.
      // (After the last tile that is the same tile again, from the caches.)
      while (true) {
        f32x4_t s[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][0] = s[mt][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        from_here(k.w);
        from_here(k.s);
        int passes = passes_of(k.w, k.s);
        for (int pass = 0;;) {
          scores(k, q, pass, passes, s);
          if (FMT != FMT_NVFP4 || ++pass >= passes) break;
        }
        load_k(k, next, ahead);
        const int beyond = ahead + 4 < end ? ahead + 4 : ahead;
        const Pages after = pages_of(beyond);
        const bool all = now.there[0] && now.there[1] && (t + 1) * kTile <= w.known;    // every row attends to all of it
        uint32_t may[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) may[mt] = 0xFFu;
        if (!all) mask_scores<MT>(a, w, b, t, now.there[0], now.there[1], row_of(0), quarter, s, may);
        u32x4_t p[MT][PP];
        softmax_step<HALF, MT, PP, kTilesV>(s, a.d.scale, minus, m, l, o, p);
        from_here(v.w);
        from_here(v.s);
        if (!all || past_bf16(v)) clean(now, t, may, v);
        passes = passes_of(v.w, v.s);
        for (int pass = 0;;) {
          values(v, p, pass, passes, o);
          if (FMT != FMT_NVFP4 || ++pass >= passes) break;
        }
        t += 4;
        if (t >= end) break;
        load_v(v, next, ahead);
        now = next;
        next = after;
        ahead = beyond;
      }
    }
    join(o, m, l, whole, slot);
    return true;
  }

  // The four waves' sums joined: written as outputs, or as a part of them.
  __device__ __forceinline__ void join(f32x4_t (&o)[MT][kTilesV], float (&m)[MT], float (&l)[MT], bool whole, float* slot) {
    place();
    __syncthreads();      // q's fragments, and the last piece's sums, have been read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] = row_sum(l[mt]);
      if (quarter == 0) {
        sm.m[wave][mt * 16 + col] = m[mt];
        sm.l[wave][mt * 16 + col] = l[mt];
      }
    }
    __syncthreads();
    float* sums = reinterpret_cast<float*>(sm.big);
#pragma unroll 1
    for (int turn = 0; turn < 4 / kBuffers; ++turn) {
      if (turn > 0) __syncthreads();
      if (wave / kBuffers != turn) continue;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 16 + col;
        const float top = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
        const float keep = m[mt] == -__builtin_inff() ? (l[mt] == 0.0f ? 0.0f : l[mt])   // nothing met, or NaN alone
                                                      : __builtin_amdgcn_exp2f(m[mt] - top);
        float* row = sums + (wave % kBuffers * kRows + r) * kPad;
#pragma unroll
        for (int u = 0; u < S::VU; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < S::VC; c += 4) {
              f32x4_t x;
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = o[mt][u * S::VC + c + e][i] * keep;
              f32x4_t* at = reinterpret_cast<f32x4_t*>(row + u * 16 * S::VC + (quarter * 4 + i) * S::VC + c);
              if (turn > 0) x += *at;
              *at = x;
            }
      }
    }
    __syncthreads();
    const int rows = a.d.tokens * a.d.group, live = w.count * a.d.group;
    for (int i = wave * 64 + lane; i < kRows * (D / 8); i += kAttnThreads) {
      const int r = i / (D / 8), ch = i % (D / 8) * 8, at = tile * kRows + r;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.0f;
#pragma unroll
      for (int s = 0; s < kBuffers; ++s) {
        const float* from = sums + (s * kRows + r) * kPad + ch;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += from[e];
      }
      const u32x2_t marks = *reinterpret_cast<const u32x2_t*>(sm.nan + r * D + ch);
      if (marks.x | marks.y)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = marked_value(x[e], (e < 4 ? marks.x : marks.y) >> (e % 4 * 8) & 3u);
      const float top = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        sum += sm.l[s][r] * (sm.m[s][r] == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(sm.m[s][r] - top));
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<f32x4_t*>(slot + r * D + ch + e) = f32x4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
        if (ch == 0) {
          slot[kRows * D + r] = top;
          slot[kRows * D + kRows + r] = sum;
        }
      } else if (at < rows) {
        write_row<DT, 8>(a, row_at(at), D, ch, x, top, at < live ? sum : 0.0f);
      }
    }
  }
};

// ------------------------------------------------------- rows of its own to each wave
// The same products where there are more rows than a wave holds: the workgroup decodes a step's keys and values once, a
// quarter to each wave, into LDS as the fragments that the products take, and each wave takes all of them for 16 * MT rows
// of its own.  Decoding costs four times less a row than where each wave decodes what it reads, and needs no registers
// beside the sums.  LDS holds one step (64 KB); two workgroups of a CU take turns at decoding and products.
template <int DT, int FMT, int D, int MT, int WAVES, bool HALF>
struct SharedAttention {
  using S = Shape<FMT, D>;
  using Other = std::conditional_t<HALF && !kHalfOnly<DT, FMT>, SharedAttention<DT, FMT, D, MT, WAVES, false>, void>;
  static constexpr int QP = kQParts<DT, FMT>, PP = HALF ? 1 : kPParts<DT>, kDim = D, kType = DT;
  static constexpr int kTilesV = D / 16, kThreads = 64 * WAVES, kRows = 16 * MT * WAVES;
  static constexpr int kStep = D <= 128 ? kTile * WAVES : 4096 * WAVES / D, kTiles = kStep / kTile;
  // waves of a SIMD that the registers are kept to: two where q and the sums leave room for it
  static constexpr int kWaves = MT * (D / 8 * QP + D / 4) <= 160 ? 2 : 1;
  static constexpr int kResident = kWaves * 4 / WAVES;                 // workgroups of a CU
  static constexpr int kStart = D == 512 ? 6 : 4, kFew = 4;
  // a wave's share of a step: a tile, or of that a part:
  static constexpr int kPartsOfTile = WAVES / kTiles;
  static constexpr int kHalves = kPartsOfTile > 1 ? 1 : 2;             // halves of its positions for the keys
  static constexpr int kUnits = kPartsOfTile > 2 ? S::KU / 2 : S::KU;  // units of them
  static constexpr int VC = D / 16 < 8 ? D / 16 : 8;                   // channels of a lane for the values, of all positions
  static constexpr int VB = S::kFp8 ? VC : VC / 2, VW = VB < 4 ? 1 : VB / 4;
  static constexpr int kWords = D / 32;                                // of a row's marks
  // Parts are kept as the registers hold them, a store of 1 KB at a time (as rows it is 64 pieces of 16 bytes: [4, 8192, 512]
  // 42 us against 40, 16-token trees 100 against 96).  Four channels of a lane are too few for the joining lanes' eight.
  static constexpr bool kFragments = VC == 8;

  struct Shared {
    __attribute__((aligned(16))) u32x4_t key[kTiles][2][S::kSteps][64];
    __attribute__((aligned(16))) u32x4_t value[kTiles][kTilesV][64];
    uint32_t odd[kStep][2 * kWords];      // channels of a position whose value is +inf or NaN, then -inf or NaN
    uint32_t nan[kRows][2 * kWords];      // outputs that one reached
    int marked;                           // the step that `odd` is of
    int reached;                          // whether `nan` has marks
    int there[kTiles];                    // which halves of a tile have a page
    int again;                            // a scale was met that fp16 does not hold
    int first[kThreads];
    int sums[4];
  };

  const AttnArgs& a;
  Shared& sm;
  int lane, col, quarter;
  const int wave;
  const MinusOne minus;
  int b, kv, tile;
  Work w;

  __device__ __forceinline__ SharedAttention(const AttnArgs& args, Shared& shared)
      : a(args), sm(shared), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
    place();
  }
  __device__ __forceinline__ void place() {
    lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    col = lane & 15;
    quarter = lane >> 4;
  }
  __device__ __forceinline__ int row_of(int mt) const { return tile * kRows + (wave * MT + mt) * 16 + col; }
  __device__ __forceinline__ int64_t row_at(int r) const {
    const int i = r / a.d.group, g = r - i * a.d.group;
    return (((int64_t)b * a.d.tokens + i) * a.d.heads + kv * a.d.group + g);
  }

  // ----- this wave's quarter of a step
  __device__ __forceinline__ int my_tile(int step) const { return step * kTiles + wave / kPartsOfTile; }
  __device__ __forceinline__ int my_half() const { return kPartsOfTile > 1 ? wave % 2 : 0; }
  __device__ __forceinline__ int my_unit() const { return kPartsOfTile > 2 ? wave / 2 * kUnits : 0; }
  __device__ __forceinline__ int my_channels() const { return kPartsOfTile > 1 ? wave % kPartsOfTile : 0; }   // 128 of them
  struct Raw {
    uint32_t k[kHalves][kUnits][S::KW], ks[kHalves][kUnits][S::KS];
    uint32_t v[8][VW], vs[8];
    int page[2], next[2];       // of the halves' positions, -1 for none; and of those of the step after
  };
  __device__ __forceinline__ void look_up(int (&page)[2], int step) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = (my_tile(step) * kTile + h * 16) >> a.d.page_shift;
      const int entry = uniform_load(a.table, (int64_t)b * a.d.width + min(slot, a.d.width - 1));
      page[h] = slot < a.d.width && (uint32_t)entry < (uint32_t)a.d.pages ? entry : -1;
    }
  }
  // The step's rows, whose pages were looked up a step ago.
  __device__ __forceinline__ void load(Raw& x, int step) const {
    const int t = my_tile(step), blocks = D >> a.block_shift;
    int64_t row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.page[h] = x.next[h];
      row[h] = (((int64_t)max(x.page[h], 0) * a.d.kv_heads + kv) << a.d.page_shift) +
               ((t * kTile + h * 16) & ((1 << a.d.page_shift) - 1));
    }
    look_up(x.next, step + 1);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int64_t r = kHalves == 2 ? row[h] : my_half() ? row[1] : row[0];
      const uint8_t* codes = a.k_codes + r * S::kRowBytes + my_unit() * S::KW * 16;
      const uint8_t* scales = a.k_scales + r * blocks;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint8_t* at = codes + (uint32_t)(col * S::kRowBytes + quarter * S::KW * 4) + u * S::KW * 16;
        if constexpr (S::KW == 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at);
          x.k[h][u][0] = v.x; x.k[h][u][1] = v.y; x.k[h][u][2] = v.z; x.k[h][u][3] = v.w;
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at);
          x.k[h][u][0] = v.x; x.k[h][u][1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < S::KS; ++i)
          x.ks[h][u][i] =
              scales[(uint32_t)(col * blocks + ((((my_unit() + u) * 4 + quarter) * S::KC + i * 16) >> a.block_shift))];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* codes = a.v_codes + row[j / 4] * S::kRowBytes + my_channels() * 16 * VB;
      const uint8_t* scales = a.v_scales + (row[j / 4] + j % 4) * blocks;
      const uint8_t* at = codes + (uint32_t)(quarter * 4 * S::kRowBytes + col * VB) + j % 4 * S::kRowBytes;
      if constexpr (VB == 2) x.v[j][0] = *reinterpret_cast<const uint16_t*>(at);
      else if constexpr (VB == 4) x.v[j][0] = *reinterpret_cast<const uint32_t*>(at);
      else {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at);
        x.v[j][0] = v.x; x.v[j][1] = v.y;
      }
      x.vs[j] = scales[(uint32_t)(quarter * 4 * blocks + ((my_channels() * 128 + col * VC) >> a.block_shift))];
    }
  }
  // Two channels in bf16; a scale that is more than its exponent is multiplied in fp32 (exact, as the product is in bf16).
  template <bool EXACT, bool TO_HALF, int I>
  __device__ __forceinline__ static uint32_t decode(const uint32_t* words, float s) {
    if constexpr (!EXACT) return decode_value<TO_HALF, FMT, I>(words, s);
    const uint32_t v = decode_pair<FMT, I>(words, 1.0f);
    const float lo = bf16_lo(v) * s, hi = bf16_hi(v) * s;
    if constexpr (TO_HALF) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, f16x2_t));
    return pack_bf16(lo, hi);
  }
  // Whether a value of the wave's part of the step may be infinite in bf16.  (Where fp16 is tried, such a scale starts the
  // piece again.)
  __device__ __forceinline__ static bool past_bf16(const Raw& x) {
    if constexpr (HALF || FMT == FMT_NVFP4) return false;
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, x.vs[j]);
    return __ballot(most >= kPastBf16<FMT>) != 0;
  }
  // Raw to LDS; positions that are none become 0, and values that are not finite, in tiles that are attended to in part or
  // hold infinities, too, with a mark.
  __device__ __forceinline__ void decode_step(Raw& x, int step, int tag) const {
    const int t = my_tile(step);
    from_here(x.k);
    from_here(x.ks);
    from_here(x.v);
    from_here(x.vs);
    if (lane == 0) sm.there[wave / kPartsOfTile] = (int)(x.page[0] >= 0) + 2 * (int)(x.page[1] >= 0);   // each part says the same
    if (!(x.page[0] >= 0 && x.page[1] >= 0 && (t + 1) * kTile <= w.known) || past_bf16(x)) clean(x, t, tag);
    if constexpr (HALF && !kHalfOnly<DT, FMT>) {
      uint32_t least = 255, most = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        least = min(least, x.vs[j]);
        most = max(most, x.vs[j]);
      }
      if (__ballot(!fits_half<FMT>(least, most)) != 0 && lane == 0) sm.again = 1;
    }
    if constexpr (FMT == FMT_NVFP4) {
      bool any = false;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
          for (int i = 0; i < S::KS; ++i) any |= beyond_exponent(scale_value<FMT>(x.ks[h][u][i]));
#pragma unroll
      for (int j = 0; j < 8; ++j) any |= beyond_exponent(scale_value<FMT>(x.vs[j]));
      if (__ballot(any) != 0) return emit<true>(x);
    }
    emit<false>(x);
  }
  template <bool EXACT>
  __device__ __forceinline__ void emit(const Raw& x) const {
    const int slot = wave / kPartsOfTile;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      static_for<kUnits>([&](auto U) {
        constexpr int u = decltype(U)::value;
        float sc[S::KS];
#pragma unroll
        for (int i = 0; i < S::KS; ++i) sc[i] = scale_operand<FMT>(x.ks[h][u][i]);
        static_for<S::kHalves>([&](auto H) {
          constexpr int hf = decltype(H)::value, is = hf / 2 < S::KS ? hf / 2 : 0;
          uint32_t y[4];
          static_for<4>([&](auto I) {
            y[decltype(I)::value] = decode<EXACT, kHalfKeys<DT, FMT>, hf * 4 + decltype(I)::value>(x.k[h][u], sc[is]);
          });
          sm.key[slot][kHalves == 2 ? h : my_half()][(my_unit() + u) * S::kHalves + hf][lane] = u32x4_t{y[0], y[1], y[2], y[3]};
        });
      });
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = scale_operand<FMT>(x.vs[j]);
    static_for<VC / 2>([&](auto I) {
      constexpr int i = decltype(I)::value;
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = decode<EXACT, HALF, i>(x.v[j], sc[j]);
      uint32_t z[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[0][j] = __builtin_amdgcn_perm(y[2 * j + 1], y[2 * j], 0x05040100u);
        z[1][j] = __builtin_amdgcn_perm(y[2 * j + 1], y[2 * j], 0x07060302u);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
        sm.value[slot][my_channels() * 8 + 2 * i + half][lane] = u32x4_t{z[half][0], z[half][1], z[half][2], z[half][3]};
    });
  }
  __device__ __forceinline__ void clean(Raw& x, int t, int tag) const {
    using Codes = Odd<FMT>;
    constexpr uint32_t kUnit = FMT == FMT_NVFP4 ? 0x38u : 127u;        // a scale of 1
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pos = t * kTile + (j / 4) * 16 + quarter * 4 + j % 4;
      const bool none = x.page[j / 4] < 0 || pos >= w.end;
      x.vs[j] = none ? kUnit : x.vs[j];
      const uint32_t more = (Codes::kHalf - least_odd<FMT>(x.vs[j])) * Codes::kOnes;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        x.v[j][i] = none ? 0u : x.v[j][i];
        any |= (x.v[j][i] & ~Codes::kTop) + more;
      }
    }
    if (__ballot((any & Codes::kTop) != 0) == 0) return;
    if (lane == 0) sm.marked = tag;
    const int channel = my_channels() * 128 + col * VC;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {          // a position at a time, its values first in line
      const int least = least_odd<FMT>(x.vs[0]);
      const uint32_t more = (Codes::kHalf - least) * Codes::kOnes;
      const int row = wave / kPartsOfTile * kTile + (j / 4) * 16 + quarter * 4 + j % 4;
#pragma unroll 1
      for (int sign = 0; sign < 2; ++sign) {
        uint32_t odd[VW], bits = 0;
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          const Codes f(x.v[0][i], more, least == 0);
          odd[i] = sign ? f.sign[1] : f.sign[0];
        }
#pragma unroll
        for (int c = 0; c < VC; ++c)
          bits |= (odd[c * Codes::kBits / 32] >> (c * Codes::kBits % 32 + Codes::kBits - 1) & 1u) << c;
        if (bits) atomicOr(&sm.odd[row][sign * kWords + channel / 32], bits << (channel % 32));
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) x.v[0][i] &= ~Codes(x.v[0][i], more, least == 0).codes();
      x.vs[0] = least == 0 ? kUnit : x.vs[0];
      to_the_end(x.v);
      to_the_end(x.vs);
    }
  }

  // Steps [first, last) of the problem; `whole`: they are all, else the sums go to `slot`.  False, with nothing written,
  // where fp16 does not hold the values.
  __device__ __forceinline__ bool piece(int first, int last, bool whole, float* slot) {
    place();
    for (int i = wave * 64 + lane; i < 2 * kRows * kWords; i += kThreads) sm.nan[i / (2 * kWords)][i % (2 * kWords)] = 0;
    clear_odd();
    if (wave == 0 && lane == 0) {
      sm.marked = -1;
      sm.reached = 0;
      sm.again = 0;
    }
    Raw x;
    look_up(x.next, first);
    bf16x8_t q[MT][S::kSteps][QP];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        const int ch = st / S::kHalves * 4 * S::KC + quarter * S::KC + st % S::kHalves * 8, r = row_of(mt);
        float e[8] = {};
        if (r < a.d.tokens * a.d.group) to_f32<DT>(load8<DT>(a.q, row_at(r) * D + ch, 8), e);
        if (a.d.negative)
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = -e[i];
        parts_of<DT, FMT>(e, minus, q[mt][st]);
      }
    f32x4_t o[MT][kTilesV];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < kTilesV; ++t) o[mt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[mt] = -__builtin_inff();
      l[mt] = 0.0f;
    }
    // waves whose rows are all padding only decode
    const bool works = tile * kRows + wave * MT * 16 < w.count * a.d.group;
    if (first < last) {
      load(x, first);
      from_here(x.ks);                     // as words, as the loads of the other variant's first tile
      from_here(x.vs);
      bool odd = false;
      for (int step = first; step < last; ++step) {
        __syncthreads();                   // the fragments of the step before have been read
        if (odd) {
          clear_odd();
          __syncthreads();
        }
        decode_step(x, step, step);
        __syncthreads();
        if (HALF && !kHalfOnly<DT, FMT> && __builtin_amdgcn_readfirstlane(sm.again)) return false;
        odd = __builtin_amdgcn_readfirstlane(sm.marked) == step;
        if (step + 1 < last) load(x, step + 1);
        if (works) products(step, q, odd, m, l, o);
      }
    }
    finish(o, m, l, whole, slot);
    return true;
  }
  __device__ __forceinline__ void clear_odd() const {
    for (int i = wave * 64 + lane; i < 2 * kStep * kWords; i += kThreads) sm.odd[i / (2 * kWords)][i % (2 * kWords)] = 0;
  }
  __device__ __forceinline__ void products(int step, const bf16x8_t (&q)[MT][S::kSteps][QP], bool odd, float (&m)[MT],
                                           float (&l)[MT], f32x4_t (&o)[MT][kTilesV]) const {
#pragma unroll 1
    for (int ti = 0; ti < kTiles; ++ti) {
      const int t = step * kTiles + ti;
      if (t * kTile >= w.end) break;
      f32x4_t s[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][0] = s[mt][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        bf16x8_t key[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) key[h] = __builtin_bit_cast(bf16x8_t, sm.key[ti][h][st][lane]);
#pragma unroll
        for (int p = 0; p < QP; ++p)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) s[mt][h] = mfma_key<kHalfKeys<DT, FMT>>(key[h], q[mt][st][p], s[mt][h]);
      }
      const int there = __builtin_amdgcn_readfirstlane(sm.there[ti]);
      if (odd || there != 3 || (t + 1) * kTile > w.known) {
        uint32_t may[MT];
        mask_scores<MT>(a, w, b, t, there & 1, there >> 1, row_of(0), quarter, s, may);
        if (odd) {
          uint32_t sees = 0;               // a bit for each row and position
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sees |= may[mt] << (8 * mt);
#pragma unroll 1
          for (int i = 0; i < 8 * MT * 2 * kWords; ++i) {
            const int at = i / (2 * kWords), word = i % (2 * kWords), j = at % 8;
            if (!(sees >> at & 1)) continue;
            const uint32_t bits = sm.odd[ti * kTile + (j / 4) * 16 + quarter * 4 + j % 4][word];
            if (bits) {
              atomicOr(&sm.nan[(wave * MT + at / 8) * 16 + col][word], bits);
              sm.reached = 1;
            }
          }
        }
      }
      u32x4_t p[MT][PP];
      softmax_step<HALF, MT, PP, kTilesV>(s, a.d.scale, minus, m, l, o, p);
#pragma unroll
      for (int t = 0; t < kTilesV; t += 2) {
        u32x4_t val[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) val[h] = sm.value[ti][t + h][lane];
#pragma unroll
        for (int part = 0; part < PP; ++part)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][t + h] = mfma_value<HALF>(val[h], p[mt][part], o[mt][t + h]);
      }
    }
  }
  __device__ __forceinline__ void finish(f32x4_t (&o)[MT][kTilesV], float (&m)[MT], float (&l)[MT], bool whole, float* slot) {
    place();
    __syncthreads();                       // the marks are all there
    const int rows = a.d.tokens * a.d.group, live = w.count * a.d.group;
    if (__builtin_amdgcn_readfirstlane(sm.reached)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < kTilesV / VC; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* marks = sm.nan[(wave * MT + mt) * 16 + col];
            const int ch = u * 16 * VC + (quarter * 4 + i) * VC;
            const uint32_t up = marks[ch / 32] >> (ch % 32), down = marks[kWords + ch / 32] >> (ch % 32);
#pragma unroll
            for (int e = 0; e < VC; ++e)
              o[mt][u * VC + e][i] = marked_value(o[mt][u * VC + e][i], (up >> e & 1u) + 2 * (down >> e & 1u));
          }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float sum = row_sum(l[mt]);
      const int r = (wave * MT + mt) * 16 + col, at = tile * kRows + r;
#pragma unroll
      for (int u = 0; u < kTilesV / VC; ++u) {
        const int ch = u * 16 * VC + quarter * 4 * VC;                   // four times VC channels
        if (!whole && kFragments) {
#pragma unroll
          for (int e = 0; e < VC; ++e)
            *reinterpret_cast<f32x4_t*>(slot + (((wave * MT + mt) * kTilesV + u * VC + e) * 64 + lane) * 4) =
                o[mt][u * VC + e];
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[VC];
#pragma unroll
          for (int e = 0; e < VC; ++e) x[e] = o[mt][u * VC + e][i];
          if (!whole) {
#pragma unroll
            for (int e = 0; e < VC; e += 4)
              *reinterpret_cast<f32x4_t*>(slot + r * D + ch + i * VC + e) = f32x4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
          } else if (at < rows) {
            write_row<DT, VC>(a, row_at(at), D, ch + i * VC, x, m[mt], at < live ? sum : 0.0f);
          }
        }
      }
      if (!whole && quarter == 0) {
        slot[kRows * D + r] = m[mt];
        slot[kRows * D + kRows + r] = sum;
      }
    }
  }
};

// Sum of v over the threads below this one, of 64 * WAVES; all of them in `total`.
template <int WAVES>
__device__ __forceinline__ int attn_scan(int v, int* sums, int& total) {
  int x = v;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int y = __shfl_up(x, s);
    if ((int)(threadIdx.x & 63) >= s) x += y;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = x;
  __syncthreads();
  int below = x - v;
  total = 0;
#pragma unroll
  for (int s = 0; s < WAVES; ++s) {
    if (s < (int)(threadIdx.x >> 6)) below += sums[s];
    total += sums[s];
  }
  return below;
}

// A piece, with fp16 probabilities where they are enough.
template <class A>
__device__ __forceinline__ void work_on(const AttnArgs& a, typename A::Shared& sm, int b, int kv, int tile, const Work& w,
                                        int first, int last, bool whole, float* slot) {
  A x(a, sm);
  x.b = b;
  x.kv = kv;
  x.tile = tile;
  x.w = w;
  if (x.piece(first, last, whole, slot)) return;
  if constexpr (!std::is_same_v<typename A::Other, void>) {
    __syncthreads();
    typename A::Other y(a, reinterpret_cast<typename A::Other::Shared&>(sm));
    y.b = b;
    y.kv = kv;
    y.tile = tile;
    y.w = w;
    y.piece(first, last, whole, slot);
  }
}

// One workgroup for each problem, in rows of kGridRow: a grid's first size times the threads has to stay below 2^32, and there
// may be 2^31 problems.
constexpr int64_t kGridRow = int64_t(1) << 20;
template <class A>
__global__ void __launch_bounds__(A::kThreads, A::kWaves) k_cache_attention(AttnArgs a) {
  __shared__ typename A::Shared sm;
  const uint32_t at = blockIdx.y * gridDim.x + blockIdx.x, each = a.d.kv_heads * a.d.row_tiles;
  const int b = at / each, kv = (at - b * each) / a.d.row_tiles, tile = at % a.d.row_tiles;
  if (b >= a.d.sequences) return;          // the last row's rest
  const Work w = work_of_all<A>(a, b);
  work_on<A>(a, sm, b, kv, tile, w, 0, tile < w.tiles ? w.steps : 0, true, nullptr);
}

// The steps of all problems shared out evenly: workgroup w takes those of share_of, a piece of a problem at a time.  A
// problem that lies within one share is written here, the others' parts are joined by k_cache_attention_join.
template <class A>
__global__ void __launch_bounds__(A::kThreads, A::kWaves) k_cache_attention_split(AttnArgs a) {
  __shared__ typename A::Shared sm;
  int total = 0;
  for (int b0 = 0; b0 < a.d.sequences; b0 += A::kThreads) {
    int sum;
    attn_scan<A::kThreads / 64>(units_of<A>(a, b0 + (int)threadIdx.x), sm.sums, sum);
    total += sum;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  const int g = min(a.d.workgroups, total), me = blockIdx.x;
  if (me >= g) return;
  int u = share_of(me, total, g);
  const int end = share_of(me + 1, total, g);
  int base = 0;                     // steps of the sequences before b0
  for (int b0 = 0; u < end; b0 += A::kThreads) {
    int sum;
    const int below = attn_scan<A::kThreads / 64>(units_of<A>(a, b0 + (int)threadIdx.x), sm.sums, sum);
    sum = __builtin_amdgcn_readfirstlane(sum);
    sm.first[threadIdx.x] = base + below;
    __syncthreads();
    while (u < min(end, base + sum)) {
      int lo = 0;                   // the last sequence of the chunk that starts at or before u, and is not empty
      for (int s = A::kThreads / 2; s > 0; s /= 2)
        if (__builtin_amdgcn_readfirstlane(sm.first[lo + s]) <= u) lo += s;
      const int seq = b0 + lo;
      const Work w = work_of_all<A>(a, seq);
      const int each = w.steps + A::kStart;
      const int local = u - __builtin_amdgcn_readfirstlane(sm.first[lo]), problem = local / each;
      const int from = local - problem * each, n = min(each - from, end - u), kv = problem / w.tiles;
      const int step = max(from - A::kStart, 0), last = from + n - A::kStart;
      if (last > step) {
        work_on<A>(a, sm, seq, kv, problem - kv * w.tiles, w, step, last, last - step == w.steps,
                   a.parts + (2 * me + (step == 0)) * kSlotFloats<A>);
        __syncthreads();
      }
      u += n;
    }
    base += sum;
    __syncthreads();
  }
}

// The parts of problems that several workgroups worked on; and zeros for those that none did.  A workgroup takes 64 groups
// of 8 channels, a lane each, and its waves take turns at the parts, so that a wave has a few parts' loads under way at a
// time (a lane that took them one after another made 12 us of 16 parts).
template <class A>
__global__ void __launch_bounds__(kAttnThreads) k_cache_attention_join(AttnArgs a) {
  constexpr int D = A::kDim;
  __shared__ int counts[4][2];
  __shared__ float sums[4][64][10];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int each = a.d.kv_heads * a.d.row_tiles;
  const int b = blockIdx.x / each, kv = (blockIdx.x - b * each) / a.d.row_tiles, tile = blockIdx.x % a.d.row_tiles;
  int before = 0, all = 0;
  for (int s = threadIdx.x; s < a.d.sequences; s += kAttnThreads) {
    const int units = units_of<A>(a, s);
    all += units;
    before += s < b ? units : 0;
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    all += __shfl_xor(all, s);
    before += __shfl_xor(before, s);
  }
  if (lane == 0) {
    counts[wave][0] = all;
    counts[wave][1] = before;
  }
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(counts[0][0] + counts[1][0] + counts[2][0] + counts[3][0]);
  int first = __builtin_amdgcn_readfirstlane(counts[0][1] + counts[1][1] + counts[2][1] + counts[3][1]);
  const Work w = work_of_all<A>(a, b);
  const int rows = a.d.tokens * a.d.group, live = w.count * a.d.group;
  const bool none = w.steps == 0 || tile >= w.tiles;
  int w0 = 0, w1 = -1;
  const int g = min(a.d.workgroups, total);
  if (!none) {
    first += (kv * w.tiles + tile) * (w.steps + A::kStart) + A::kStart;
    w0 = owner_of(first, total, g);
    w1 = owner_of(first + w.steps - 1, total, g);
    if (w0 == w1) return;
  }
  int r = blockIdx.y * (512 / D) + lane / (D / 8), ch = lane % (D / 8) * 8, from = r * D + ch;
  if constexpr (A::kFragments) {
    // the same 64 groups of 16 rows and 32 channels (a quarter's), where SharedAttention::finish puts them
    const int piece = blockIdx.y / (D / 32), u = blockIdx.y % (D / 32) / 4, quarter = blockIdx.y % 4;
    r = piece * 16 + lane / 4;
    ch = u * 128 + (quarter * 4 + lane % 4) * 8;
    from = ((piece * (D / 16) + u * 8) * 64 + quarter * 16) * 4 + lane;
  }
  const int at = tile * A::kRows + r;
  const bool wanted = at < rows;
  float x[8] = {}, top = -__builtin_inff(), sum = 0.0f;
  if (wanted && at < live) {
    auto slot_of = [&](int s) { return a.parts + (int64_t)(2 * s + (s == w0)) * kSlotFloats<A>; };
#pragma unroll 4
    for (int s = w0 + wave; s <= w1; s += 4) top = fmaxf(top, slot_of(s)[A::kRows * D + r]);
#pragma unroll 2
    for (int s = w0 + wave; s <= w1; s += 4) {
      const float* slot = slot_of(s);
      const float m = slot[A::kRows * D + r], l = slot[A::kRows * D + A::kRows + r];
      f32x4_t lo, hi;
      if constexpr (A::kFragments) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = slot[from + e * 256];
          hi[e] = slot[from + e * 256 + 1024];
        }
      } else {
        lo = *reinterpret_cast<const f32x4_t*>(slot + from);
        hi = *reinterpret_cast<const f32x4_t*>(slot + from + 4);
      }
      const float keep = share_of_part(m, l, top);
      sum += m == -__builtin_inff() ? l : l * keep;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] += lo[e] * keep;
        x[4 + e] += hi[e] * keep;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[wave][lane][e] = x[e];
  sums[wave][lane][8] = top;
  sums[wave][lane][9] = sum;
  __syncthreads();
  if (wave != 0 || !wanted) return;
  float best = -__builtin_inff(), whole = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s) best = fmaxf(best, sums[s][lane][8]);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float m = sums[s][lane][8], l = sums[s][lane][9];
    const float keep = share_of_part(m, l, best);
    whole += m == -__builtin_inff() ? l : l * keep;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += sums[s][lane][e] * keep;
  }
  const int t = at / a.d.group;
  write_row<A::kType, 8>(a, ((int64_t)b * a.d.tokens + t) * a.d.heads + kv * a.d.group + (at - t * a.d.group), D, ch, x, best,
                         whole);
}

// Rows of a problem's tile.  Up to 16 or 32: the four waves take different positions of the same rows, so that a few rows
// keep a whole workgroup's loads under way (32 sequences of 8192 with 32 rows 76 us, 89 the other way).  More: each wave has
// rows of its own, 32 (16 of the wide heads), and all take the same positions, decoded once (64 rows 164 us with the first
// way, 143 so); two waves are enough for 64 (four, half of them idle, 121 us against 118).
inline int attention_rows(int dim, int64_t rows) {
  if (rows <= 16) return 16;
  if (rows <= 32 && dim <= 128) return 32;
  return rows <= 64 || dim > 128 ? 64 : 128;
}
template <int DT, int FMT, int D, int ROWS>
struct KernelOf {
  using Type = std::conditional_t<
      (ROWS <= 32), Attention<DT, FMT, D, (ROWS <= 32 ? ROWS / 16 : 1), kHalfOnly<DT, FMT>>,
      SharedAttention<DT, FMT, D, (D <= 128 ? 2 : 1), (ROWS == 64 && D <= 128 ? 2 : 4),
                      (kHalfOnly<DT, FMT> || (DT == DT_BF16 && D <= 256))>>;
};
// What the launches have to know of a kernel.
struct AttnShape {
  int step, start, few, resident;   // positions of a step; units before a problem's steps; kFew; workgroups of a CU
};

template <class A>
hipError_t launch_attention_of(const AttnArgs& a, int64_t problems, hipStream_t st) {
  if (a.d.workgroups == 0) {
    const dim3 grid((unsigned)min(problems, kGridRow), (unsigned)((problems + kGridRow - 1) / kGridRow));
    k_cache_attention<A><<<grid, A::kThreads, 0, st>>>(a);
  } else {
    k_cache_attention_split<A><<<(unsigned)a.d.workgroups, A::kThreads, 0, st>>>(a);
    k_cache_attention_join<A><<<dim3((unsigned)problems, A::kRows * A::kDim / 512), kAttnThreads, 0, st>>>(a);
  }
  return hipGetLastError();
}

// The kernel for a head size and rows: its shape (a NULL), or a launch.
template <int DT, int FMT>
hipError_t attention_dim(const AttnArgs* a, int dim, int rows, int64_t problems, AttnShape* shape, hipStream_t st) {
#define CASE(D, ROWS)                                         \
  if (dim == D && rows == ROWS) {                             \
    using A = typename KernelOf<DT, FMT, D, ROWS>::Type;      \
    if (a) return launch_attention_of<A>(*a, problems, st);   \
    *shape = {A::kStep, A::kStart, A::kFew, A::kResident};    \
    return hipSuccess;                                        \
  }
  CASE(64, 16)
  CASE(64, 32)
  CASE(64, 64)
  CASE(64, 128)
  CASE(128, 16)
  CASE(128, 32)
  CASE(128, 64)
  CASE(128, 128)
  CASE(256, 16)
  CASE(256, 64)
  CASE(512, 16)
  CASE(512, 64)
#undef CASE
  return hipErrorInvalidValue;
}

// The kernels of one type and format (csrc/cache_attention_<format>_<type>.hip).
template <int DT, int FMT>
hipError_t attention_kernels(const AttnArgs* a, int dim, int rows, int64_t problems, AttnShape* shape, hipStream_t st);
#define DECLARE(DT, FMT)                                                                                               \
  template <>                                                                                                          \
  hipError_t attention_kernels<DT, FMT>(const AttnArgs* a, int dim, int rows, int64_t problems, AttnShape* shape, hipStream_t st)
#define DECLARE_FORMATS(DT) \
  DECLARE(DT, FMT_FP8);     \
  DECLARE(DT, FMT_MXFP4);   \
  DECLARE(DT, FMT_NVFP4)
DECLARE_FORMATS(DT_F32);
DECLARE_FORMATS(DT_BF16);
DECLARE_FORMATS(DT_F16);
#undef DECLARE_FORMATS
#undef DECLARE

}  // namespace mxq
