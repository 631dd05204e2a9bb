// The router: scores, balance bias, expert groups, top-k and weights
// (moe_route), and the weights' gradient with respect to the logits.
//
// Which expert comes next may hang on keys that fp32 does not tell apart, so the
// choice is made on fp64 keys, ties to the lower index -- but an fp64
// exponential for every expert costs more than all the rest.  So the kernels
// compute fp32 keys, whose error is bounded (key_error), take as candidates
// every expert that the bound leaves in the running for the top_k (a few more
// than top_k), and give each candidate a lane, an fp64 key and a rank: the
// number of candidates before it.  Three kernels, chosen by what fits:
//   k_moe_route_rows     16 lanes a token: up to 512 experts, 16 places, up to 16
//                        groups, a group as whole lanes of up to 32 experts;
//   k_moe_route          a wave a token: up to 1024 experts, 32 places, groups of
//                        whole lanes (of 1, 2, 4, 8 or 16 experts);
//   k_moe_route_general  a wave a token with fp64 keys in LDS throughout: any
//                        group size.
// 16384 tokens x 256 experts, 8 of 256 in 4 of 8 groups, sigmoid and bias, fp32:
// 10.2, 23.8 and 50.6 us.  In the first a wave of four tokens runs through some 860
// vector instructions, most of them waiting for the one before (loads, halvings
// that count by ballots, the candidates through LDS, fp64 scores, ranks): four
// tokens alone take 4.6 us, and 65536 take 25.3, 0.31 ns for each one more, where
// its logits take 0.21 ns at a copy's rate.
//
// To close an expert, a bias of -inf costs nothing.  A large finite one (-1e9, the
// type's lowest) lends its rounding error to the bound that tells groups apart:
// with a whole group closed so, every token's groups are looked at again in fp64
// (16384 tokens 21.4 us and 10.0 with -inf; 64 tokens 15.1 and 4.9).
#include "moe_launch.hpp"
#include "moe_device.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 64;   // per workgroup

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// -inf and NaN logits make an expert ineligible.
__device__ __forceinline__ bool eligible(float x) { return x > -INFINITY; }

__device__ __forceinline__ double sigmoid_f64(double x) {
  const double a = exp(-fabs(x));
  return (x >= 0.0 ? 1.0 : a) / (1.0 + a);
}

// The wave's largest (key, lowest index on ties); index -1 if every key is -inf.
__device__ __forceinline__ void wave_argmax(double& key, int& at) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double k = __shfl_xor(key, d);
    const int a = __shfl_xor(at, d);
    if (k > key || (k == key && (unsigned)a < (unsigned)at)) { key = k; at = a; }
  }
}

// One token by one wave; key: experts doubles of the wave's own LDS.
template <int DT>
__device__ void route_token(const RouteArgs& a, int64_t token, double* key) {
  const int lane = threadIdx.x & 63, E = a.experts;
  const uint8_t* x = (const uint8_t*)a.logits + token * E * kElemBytes<DT>;
  const bool alive = !a.token_mask || a.token_mask[token];
  // softmax statistics over the eligible experts
  float top = -INFINITY;
  double z = 1.0;
  if (!a.sigmoid && alive) {
    for (int e = lane; e < E; e += 64) {
      const float v = elem_value<DT>(load_bits<DT>(x + e * kElemBytes<DT>));
      if (eligible(v)) top = fmaxf(top, v);
    }
    top = wave_max(top);
    double s = 0.0;
    for (int e = lane; e < E; e += 64) {
      const float v = elem_value<DT>(load_bits<DT>(x + e * kElemBytes<DT>));
      if (eligible(v)) s += exp((double)v - (double)top);
    }
    z = wave_sum(s);
  }
  auto score = [&](float v) { return a.sigmoid ? sigmoid_f64((double)v) : exp((double)v - (double)top) / z; };
  const bool by_logit = !a.bias && a.groups == 1;
  if (alive)
    for (int e = lane; e < E; e += 64) {
      const float v = elem_value<DT>(load_bits<DT>(x + e * kElemBytes<DT>));
      double k = -INFINITY;
      if (eligible(v)) {
        k = by_logit ? (double)v : score(v) + (a.bias ? (double)a.bias[e] : 0.0);
        if (!(k > -INFINITY)) k = -INFINITY;
      }
      key[e] = k;
    }
  wave_sync();
  if (alive && a.groups > 1) {
    const int size = E / a.groups;
    double best = -INFINITY, second = -INFINITY;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double k = key[lane * size + i];
        if (k > best) { second = best; best = k; }
        else if (k > second) second = k;
      }
    const double value = a.group_best == 2 && second > -INFINITY ? best + second : best;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double v = __shfl(value, g);
      rank += v > value || (v == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
    wave_sync();
    for (int e = lane; e < E; e += 64)
      if (!((kept >> (e / size)) & 1)) key[e] = -INFINITY;
    wave_sync();
  }
  // lane j keeps the j-th choice
  int mine = -1;
  if (alive)
    for (int j = 0; j < a.top_k; ++j) {
      double k = -INFINITY;
      int at = -1;
      for (int e = lane; e < E; e += 64)
        if (key[e] > k) { k = key[e]; at = e; }
      wave_argmax(k, at);
      if (at < 0) break;
      if (lane == j) mine = at;
      wave_sync();
      if (lane == 0) key[at] = -INFINITY;
      wave_sync();
    }
  float logit = -INFINITY;
  if (mine >= 0) logit = elem_value<DT>(load_bits<DT>(x + mine * kElemBytes<DT>));
  double s = 0.0;
  if (!a.sigmoid && a.renormalize) {
    const float most = wave_max(logit);              // the chosen scores up to a common factor, none vanishing
    if (mine >= 0) s = exp((double)logit - (double)most);
  } else if (mine >= 0) {
    s = score(logit);
  }
  double w = a.scale * s;
  if (a.renormalize) {
    const double sum = wave_sum(s);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.top_k) {
    a.index[token * a.top_k + lane] = mine;
    a.weights[token * a.top_k + lane] = mine >= 0 ? (float)w : 0.0f;
  }
  wave_sync();
}

template <int DT>
__global__ void __launch_bounds__(kThreads) k_moe_route_general(RouteArgs a) {
  extern __shared__ double keys[];
  const int wave = threadIdx.x >> 6;
  const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
  if (token < a.tokens) route_token<DT>(a, token, keys + wave * a.experts);
}

// ------------------------------------------------- fp32 keys, fp64 candidates
// fp32 score: of an exponential at full rate, as its error is bounded, not
// small.  In units of u = 2^-24 (half an ulp of 1) times the largest score there
// can be (sigmoid 1, softmax 1 / z):
// sigmoid 1 / (1 + e), e = 2^(-x log2 e): e is off by 1.4 |x| u (the product and
// the constant) and 2 u, which moves the score by s (1 - s) times that, at most
// u; the sum adds u and the reciprocal 2 u: 4.  softmax p = e / z, e = 2^((x -
// top) log2 e): p |x - top| 2.4 u <= u and 2 u, or 4 u by exp_neg; z in fp64 or a
// sum of such exponentials, 4 u; its reciprocal and the product 3 u: 11.  A bias
// adds half an ulp of the key, u times its size.
constexpr float kUlp = 0x1p-24f;
constexpr float kScoreError = 12.0f;
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLowest = -0x1.fffffep+127f;
// Finite for every finite key, biases next to the type's lowest value among them.
__device__ __forceinline__ float key_error(float key, float most) {
  return kUlp * kScoreError * most + 1.25f * kUlp * fabsf(key);
}
// The least fp32 key whose fp64 key may still be as large as that of an fp32 key
// c.  Never below the lowest finite value: -inf stands for an expert that is
// closed, or for no expert at all, whose logits must not be read.  A key of +inf
// has no error: only a bias of +inf makes one, in fp64 too.
__device__ __forceinline__ float reach_of(float c, float most) {
  return c < INFINITY ? fmaxf(c - 2.0f * key_error(c, most), kLowest) : c;
}
__device__ __forceinline__ float sigmoid_key(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}
__device__ __forceinline__ float softmax_key(float x, float top, float rz) {
  return __builtin_amdgcn_exp2f((x - top) * kLog2e) * rz;
}

template <typename T>
__device__ __forceinline__ T lane_value(T v, int lane);   // v of a lane that is the same for the whole wave
template <>
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
template <>
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
template <>
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// v of the lane that the DPP control names (one that names a lane for every
// lane: with bound_ctrl the old value does not matter, so the move folds into
// the operation that uses it).
template <int CTRL, typename T>
__device__ __forceinline__ T dpp_value(T v) {
  auto move = [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, CTRL, 0xF, 0xF, true); };
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, move(__builtin_bit_cast(uint32_t, v)));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(T, ((uint64_t)move((uint32_t)(b >> 32)) << 32) | move((uint32_t)b));
  }
}
// `op` over the wave, the same in every lane: within rows of 16 by DPP, across them by lane reads.
template <typename T, typename Op>
__device__ __forceinline__ T wave_all(T v, Op op) {
  v = op(v, dpp_value<0xB1>(v));
  v = op(v, dpp_value<0x4E>(v));
  v = op(v, dpp_value<0x141>(v));
  v = op(v, dpp_value<0x140>(v));
  return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}

// The two largest of a set of keys; adding another set's two is the union.
template <typename T>
struct Two {
  T best = -INFINITY, next = -INFINITY;
  __device__ __forceinline__ void add(T k) {       // not NaN
    if constexpr (sizeof(T) == 4) {
      next = __builtin_amdgcn_fmed3f(best, next, k);
      best = fmaxf(best, k);
    } else {
      next = k > best ? best : (k > next ? k : next);
      best = k > best ? k : best;
    }
  }
};

// A group's value (half of it in fp32: see group_value), a bound on its error
// where its keys are fp32 ones, and the smallest key in it.
template <typename T>
struct GroupValue {
  T value;
  float error;
  T least;
};

union GroupPairs {
  float f[128];
  double d[128];
};

// Value of the group that this lane's experts belong to, the same in every
// lane of the group: its `best` (1 or 2) largest keys summed.  t: the two
// largest of this lane's keys; lanes: lanes of a group, 32 at most (there are two
// groups or more); lds: the wave's own;
// the token's lanes are those from `base` to `end`; most: the largest score there can be.
template <typename T>
__device__ __forceinline__ GroupValue<T> group_value(Two<T> t, int lanes, int best, T* lds, int base, int end,
                                                     float most) {
  const int lane = threadIdx.x & 63;
  if ((lanes & (lanes - 1)) == 0) {
    auto meet = [&](T b, T n) { t.add(b); t.add(n); };
    if (lanes > 1) meet(dpp_value<0xB1>(t.best), dpp_value<0xB1>(t.next));
    if (lanes > 2) meet(dpp_value<0x4E>(t.best), dpp_value<0x4E>(t.next));
    if (lanes > 4) meet(dpp_value<0x141>(t.best), dpp_value<0x141>(t.next));
    if (lanes > 8) meet(dpp_value<0x140>(t.best), dpp_value<0x140>(t.next));
    if (lanes > 16) meet(__shfl_xor(t.best, 16), __shfl_xor(t.next, 16));
  } else {
    lds[2 * lane] = t.best;
    lds[2 * lane + 1] = t.next;
    wave_sync();
    const int first = base + (lane - base) / lanes * lanes;
    t = Two<T>();
    for (int i = first; i < min(end, first + lanes); ++i) {
      t.add(lds[2 * i]);
      t.add(lds[2 * i + 1]);
    }
    wave_sync();
  }
  if (!(t.best > -INFINITY)) return {t.best, 0.0f, t.best};
  const bool pair = best == 2 && t.next > -INFINITY;
  const T least = pair ? t.next : t.best;
  // a key of +inf leaves no doubt about the value: 0 for its error, so that the other groups' places do not hang on it
  if (!(t.best < INFINITY)) return {t.best, 0.0f, least};
  // The sum of two keys past half of fp32's range would be infinite, and all such groups equal: fp32 values are halved.
  const T part = sizeof(T) == 4 ? T(0.5) : T(1);
  // two keys' errors, and the sum's rounding
  const float error = pair ? 2.0f * kUlp * kScoreError * most + 2.5f * kUlp * fabsf((float)t.best) +
                                 2.5f * kUlp * fabsf((float)t.next)
                           : key_error((float)t.best, most);
  return {pair ? part * t.best + part * t.next : part * t.best, (float)part * error, least};
}

// Whether this lane's group is among the `top` groups of largest value; near:
// whether a group's place inside or outside hangs on a difference that the
// values' errors leave open.
template <typename T>
__device__ __forceinline__ bool group_kept(const GroupValue<T>& own, int groups, int lanes, int top, bool& near) {
  const int g = (threadIdx.x & 63) / lanes;
  int rank = 0;
  bool close = false;
  for (int o = 0; o < groups; ++o) {
    const T v = lane_value(own.value, o * lanes);
    const float e = lane_value(own.error, o * lanes);
    rank += v > own.value || (v == own.value && o < g);
    close |= o != g && v <= own.value && (float)(own.value - v) <= own.error + e;
  }
  near = __ballot(g < groups && rank == top - 1 && close) != 0;
  return rank < top;
}

// Logits (or biases) of experts e0 .. e0 + V - 1 of a row, of which `mine` exist; the others read as -inf.
template <int DT, int V>
__device__ __forceinline__ void load_logits(const uint8_t* row, int e0, int mine, float (&x)[V]) {
  auto four = [&](int v) {
    if constexpr (DT == DT_F32) {
      const u32x4_t w = *reinterpret_cast<const u32x4_any*>(row + (e0 + v) * 4);
      x[v] = as_f32(w.x); x[v + 1] = as_f32(w.y); x[v + 2] = as_f32(w.z); x[v + 3] = as_f32(w.w);
    } else {
      const u32x2_t w = *reinterpret_cast<const u32x2_any*>(row + (e0 + v) * 2);
      x[v] = elem_value<DT>(w.x & 0xFFFFu); x[v + 1] = elem_value<DT>(w.x >> 16);
      x[v + 2] = elem_value<DT>(w.y & 0xFFFFu); x[v + 3] = elem_value<DT>(w.y >> 16);
    }
  };
  if (V % 4 == 0 && mine == V) {
#pragma unroll
    for (int v = 0; v + 3 < V; v += 4) four(v);
    return;
  }
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    if (V % 4 == 0 && v + 4 <= mine) {
      four(v);
    } else {
#pragma unroll
      for (int i = v; i < v + 4 && i < V; ++i)
        x[i] = i < mine ? elem_value<DT>(load_bits<DT>(row + (e0 + i) * kElemBytes<DT>)) : -INFINITY;
    }
  }
}

// The keys at or above c (which is not -inf) among this lane's, bit v for key v.
template <int V>
__device__ __forceinline__ uint32_t in_reach(const float (&key)[V], float c) {
  uint32_t m = 0;
#pragma unroll
  for (int v = V - 1; v >= 0; --v) m = m + m + (key[v] >= c ? 1u : 0u);
  return m;
}

// A point between lo and hi to count at: their mean, or in every other step the
// middle of the floats between them, which comes near whatever lies far below
// hi (logits masked with the lowest value of their type) in a few steps and
// ends the halving after 64 of them.
__device__ __forceinline__ float halfway(float lo, float hi, int step) {
  if ((step & 1) == 0) return 0.5f * lo + 0.5f * hi;
  auto order = [](float f) {
    const uint32_t b = as_u32(f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  };
  const uint32_t a = order(lo), m = a + (order(hi) - a) / 2;
  return as_f32(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
}

struct Candidate {
  int expert;
  float logit;
};

// Experts lane * V .. lane * V + V - 1 in each lane; experts <= 64 V, and a
// group (if there are groups) is whole lanes.
template <int DT, int V>
__global__ void __launch_bounds__(kThreads) k_moe_route(RouteArgs a) {
  __shared__ Candidate found[kTokens][64];
  __shared__ GroupPairs pairs[kTokens];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, E = a.experts;
  const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
  if (token >= a.tokens) return;
  const bool alive = !a.token_mask || a.token_mask[token];
  const uint8_t* row = (const uint8_t*)a.logits + token * E * kElemBytes<DT>;
  const int e0 = lane * V, mine = alive ? min(V, max(0, E - e0)) : 0;

  float x[V], key[V], bias[V];
  load_logits<DT, V>(row, e0, mine, x);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.bias && v < mine ? a.bias[e0 + v] : 0.0f;
    if (!(x[v] > -INFINITY)) x[v] = -INFINITY;            // NaN too
  }
  const bool by_logit = !a.bias && a.groups == 1;
  // softmax statistics: z in fp64, as it moves every key
  float top = -INFINITY;
  double z = 1.0;
  if (!a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    top = wave_all(top, [](float p, float q) { return fmaxf(p, q); });
    if (!by_logit || !a.renormalize) {
      double s = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) s += x[v] > -INFINITY ? exp((double)x[v] - (double)top) : 0.0;
      z = wave_all(s, [](double p, double q) { return p + q; });
    }
  }
  const float rz = a.sigmoid ? 1.0f : (float)(1.0 / z);
  auto score64 = [&](float l) { return a.sigmoid ? sigmoid_f64((double)l) : exp((double)l - (double)top) / z; };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float s = by_logit ? x[v] : a.sigmoid ? sigmoid_key(x[v]) : softmax_key(x[v], top, rz);
    const float k = s + bias[v];
    key[v] = x[v] > -INFINITY && k > -INFINITY ? k : -INFINITY;
  }

  // fp64 key of this lane's expert e0 + v, read again: the rare paths below keep no registers for it
  auto key64 = [&](int v, float& l) {
    l = elem_value<DT>(load_bits<DT>(row + (e0 + v) * kElemBytes<DT>));
    const float b = a.bias ? a.bias[e0 + v] : 0.0f;
    if (!eligible(l) || !eligible(b)) return (double)-INFINITY;
    return by_logit ? (double)l : score64(l) + (double)b;
  };
  bool kept = true;
  if (a.groups > 1) {
    const int lanes = E / a.groups / V;
    Two<float> t;
#pragma unroll
    for (int v = 0; v < V; ++v) t.add(key[v]);
    bool near;
    const GroupValue<float> value = group_value<float>(t, lanes, a.group_best, pairs[wave].f, 0, 64, rz);
    kept = group_kept(value, a.groups, lanes, a.top_groups, near);
    if (near) {                        // again in fp64, from the keys that can be among a group's largest
      Two<double> t64;
      const float least = value.least > -INFINITY ? reach_of(value.least, rz) : INFINITY;
#pragma unroll 1
      for (uint32_t m = in_reach(key, least); m; m &= m - 1) {
        float l;
        t64.add(key64(__builtin_ctz(m), l));
      }
      kept = group_kept(group_value<double>(t64, lanes, a.group_best, pairs[wave].d, 0, 64, rz), a.groups, lanes,
                        a.top_groups, near);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = kept ? key[v] : -INFINITY;
  }

  // A bound `cut` with at least top_k keys at or above it and not many more:
  // halving between the smallest and the largest key.
  auto count = [&](float at) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += __popcll(__ballot(key[v] >= at));
    return n;
  };
  const int able = count(kLowest);
  float cut = kLowest;
  if (able > a.top_k + 8) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      lo = key[v] > -INFINITY ? fminf(lo, key[v]) : lo;
      hi = fmaxf(hi, key[v]);
    }
    lo = wave_all(lo, [](float p, float q) { return fminf(p, q); });
    hi = wave_all(hi, [](float p, float q) { return fmaxf(p, q); });
    cut = lo;
    for (int i = 0; i < 64; ++i) {
      const float mid = halfway(lo, hi, i);
      const int n = count(mid);
      if (n >= a.top_k) {
        cut = lo = mid;
        if (n <= a.top_k + 8) break;
      } else {
        hi = mid;
      }
    }
    if (!by_logit) cut = reach_of(cut, rz);
  }
  const int n = count(cut);

  int expert = -1;
  double k64 = -INFINITY;
  float logit = -INFINITY;
  int rank = lane;
  bool chosen = false;
  if (n <= 64) {
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t in = __ballot(key[v] >= cut);
      if (key[v] >= cut) found[wave][at + __popcll(in & ((1ull << lane) - 1))] = {e0 + v, x[v]};
      at += __popcll(in);
    }
    wave_sync();
    if (lane < n) {
      const Candidate c = found[wave][lane];
      expert = c.expert;
      logit = c.logit;
      k64 = by_logit ? (double)logit : score64(logit) + (a.bias ? (double)a.bias[expert] : 0.0);
      rank = 0;
    }
    for (int o = 0; o < n; ++o) {
      const double k = lane_value(k64, o);
      const int e = lane_value(expert, o);
      if (lane < n) rank += k > k64 || (k == k64 && e < expert);
    }
    chosen = lane < n && rank < a.top_k;
  } else {
    // More experts than lanes within the error of each other (many equal
    // logits): lane j takes the largest (key, expert) that comes after lane
    // j - 1's.  There are top_k of them, as n > 64.
    double last = INFINITY;
    int last_e = -1;
    for (int j = 0; j < a.top_k; ++j) {
      double best = -INFINITY;
      int best_e = -1;
      float best_x = 0.0f;
#pragma unroll 1
      for (int v = 0; v < (kept ? mine : 0); ++v) {
        float l;
        const double k = key64(v, l);
        if ((k < last || (k == last && e0 + v > last_e)) && k > best) { best = k; best_e = e0 + v; best_x = l; }
      }
      const double own = best;
      int at = best_e;
      wave_argmax(best, at);
      const int from = __ffsll((unsigned long long)__ballot(own == best && best_e == at && at >= 0)) - 1;
      const float l = lane_value(best_x, from);
      if (lane == j) { expert = at; logit = l; chosen = true; }
      last = best;
      last_e = at;
    }
  }
  double s = 0.0;
  if (!a.sigmoid && a.renormalize) {
    // the chosen scores up to a common factor, none vanishing
    const float most = wave_all(chosen ? logit : -INFINITY, [](float p, float q) { return fmaxf(p, q); });
    if (chosen) s = exp((double)logit - (double)most);
  } else if (chosen) {
    s = score64(logit);
  }
  double w = a.scale * s;
  if (a.renormalize) {
    const double sum = wave_all(chosen ? s : 0.0, [](double p, double q) { return p + q; });
    w = sum > 0.0 ? w / sum : 0.0;
  }
  // places without an expert: those from n on
  if (chosen || (lane >= n && lane < a.top_k)) {
    a.index[token * a.top_k + rank] = chosen ? expert : -1;
    a.weights[token * a.top_k + rank] = chosen ? (float)w : 0.0f;
  }
}

// ------------------------------------------------------ four tokens a wave
// The same for up to 512 experts and 16 places with 16 lanes a token: one
// instruction serves four tokens in what is done once a token (the fp64 scores
// of the candidates, their ranks, the groups), which is most of the work.
// Grouped sigmoid router with a bias, 256 experts, here and wave-wide: 4 tokens
// 4.7 and 5.4 us, 1024 tokens 5.3 and 6.0, 16384 tokens 10.2 and 23.8, 65536
// tokens 25.5 and 82; 512 experts, 16384 tokens 14.8 and 31.8.

// Number of set lanes of `m` in this lane's row of 16.
__device__ __forceinline__ int row_count(uint64_t m) {
  return __builtin_popcount((uint32_t)(m >> (threadIdx.x & 48)) & 0xFFFFu);
}
template <typename T, typename Op>
__device__ __forceinline__ T row_all(T v, Op op) {
  v = op(v, dpp_value<0xB1>(v));
  v = op(v, dpp_value<0x4E>(v));
  v = op(v, dpp_value<0x141>(v));
  return op(v, dpp_value<0x140>(v));
}
// Sum over the lower lanes of the row.
__device__ __forceinline__ int row_before(int v) {
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, true);
  return s - v;
}
// Value of lane `from` (0..15) of this lane's row.
template <typename T>
__device__ __forceinline__ T row_lane(T v, int from) {
  return __shfl(v, (int)(threadIdx.x & 48) + from);
}
// Rank of key among the row's: larger keys come first, equal ones in lane order.
template <int N>
__device__ __forceinline__ int row_rank(double key) {
  if constexpr (N == 0) return 0;
  else {
    const double k = dpp_value<0x120 + N>(key);       // row_ror: from lane - N
    return ((int)(k > key) | ((int)(k == key) & (int)((threadIdx.x & 15) >= N))) + row_rank<N - 1>(key);
  }
}

// Whether another lane's key is within `error` of this one's, which is finite.
template <int N>
__device__ __forceinline__ bool row_close(float key, float error) {
  if constexpr (N == 0) return false;
  else return (int)(fabsf(dpp_value<0x120 + N>(key) - key) <= error) | (int)row_close<N - 1>(key, error);
}

// How a token's experts lie in its 16 lanes: `lanes` lanes a group, `each`
// experts a lane (the last ones of a group fewer), each <= V.
struct RowLayout {
  int lanes, each;
  int inverse;   // l / lanes = l * inverse >> 8 for l < 16
};

template <int DT, int V, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) k_moe_route_rows(RouteArgs a, RowLayout in) {
  __shared__ int32_t found[kTokens][64];
  __shared__ GroupPairs pairs[kTokens];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15, E = a.experts;
  const int64_t token = ((int64_t)blockIdx.x * kTokens + wave) * 4 + (lane >> 4);
  const bool alive = token < a.tokens && (!a.token_mask || a.token_mask[token]);
  const uint8_t* row = (const uint8_t*)a.logits + token * E * kElemBytes<DT>;
  const int g = l * in.inverse >> 8, part = (l - g * in.lanes) * in.each, size = a.group_size;
  const int e0 = g * size + part, mine = alive && g < a.groups ? min(in.each, max(0, size - part)) : 0;
  constexpr float kNone = -INFINITY;

  float x[V], key[V];
  load_logits<DT, V>(row, e0, mine, x);
  const bool by_logit = !a.bias && a.groups == 1;
  // Softmax: the sum of fp32 exponentials, each off by 4 u, is enough for the
  // weights and for keys that are clear of each other; where they are not,
  // exact_z() takes its place for that token.
  float top = kNone, rz = 1.0f;
  double z = 1.0;
  if (by_logit) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = x[v];
  }
  if (SIGMOID) {
    if (!by_logit) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v] == kNone ? kNone : sigmoid_key(x[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    top = row_all(top, [](float p, float q) { return fmaxf(p, q); });
    if (!by_logit || !a.renormalize) {
      float e[V];
      double sum = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = x[v] > kNone ? exp_neg(top - x[v]) : 0.0f;
        sum += (double)e[v];
      }
      z = row_all(sum, [](double p, double q) { return p + q; });
      rz = (float)(1.0 / z);
      if (!by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = x[v] > kNone ? e[v] * rz : kNone;
      }
    }
  }
  auto exact_z = [&]() {
    double sum = 0.0;
#pragma unroll 1
    for (int v = 0; v < mine; ++v) {
      const float logit = elem_value<DT>(load_bits<DT>(row + (e0 + v) * kElemBytes<DT>));
      sum += eligible(logit) ? exp((double)logit - (double)top) : 0.0;
    }
    return row_all(sum, [](double p, double q) { return p + q; });
  };
  bool sure = SIGMOID || by_logit;     // whether z is exact, or moves no key
  auto score64 = [&](float v) { return SIGMOID ? sigmoid_f64((double)v) : exp((double)v - (double)top) / z; };
  if (!by_logit) {
    if (a.bias) {
      float b[V];
      load_logits<DT_F32, V>((const uint8_t*)a.bias, e0, mine, b);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] += b[v];
    }
  }
  // A NaN (of a logit or a bias) is no key: the median of three that Two takes is not defined for it.
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = fmaxf(key[v], kNone);
  // fp64 key of expert e of this token, its logit, and its score where the key needs that
  struct Expert {
    float logit;
    double score;
  };
  auto key64 = [&](int e, Expert& x) {
    x.logit = elem_value<DT>(load_bits<DT>(row + e * kElemBytes<DT>));
    x.score = by_logit ? 0.0 : score64(x.logit);
    const float b = a.bias ? a.bias[e] : 0.0f;
    if (!((int)eligible(x.logit) & (int)eligible(b))) return (double)-INFINITY;
    return by_logit ? (double)x.logit : x.score + (double)b;
  };

  Two<float> two;
#pragma unroll
  for (int v = 0; v < V; ++v) two.add(key[v]);
  bool kept = true;
  if (a.groups > 1) {
    const int lanes = in.lanes, base = lane & 48;
    auto keep = [&](auto own_group, bool& near) {
      int rank = 0;
      int close = 0;
      const float error = 2.0f * row_all(own_group.error, [](float p, float q) { return fmaxf(p, q); });
      for (int o = 0; o < a.groups; ++o) {
        const auto v = row_lane(own_group.value, o * lanes);
        rank += (int)(v > own_group.value) | ((int)(v == own_group.value) & (int)(o < g));
        close |= (int)(o != g) & (int)(v <= own_group.value) & (int)((float)(own_group.value - v) <= error);
      }
      near = g < a.groups && rank == a.top_groups - 1 && close;
      return rank < a.top_groups;
    };
    bool near;
    const GroupValue<float> value = group_value<float>(two, lanes, a.group_best, pairs[wave].f, base, base + 16, rz);
    kept = keep(value, near);
    if (__any(near)) {
      if (!sure) {
        const double exact = exact_z();
        const bool mine_near = row_count(__ballot(near)) > 0;   // this token's, not its neighbours' in the wave
        z = mine_near ? exact : z;
        sure = mine_near;
      }
      Two<double> t64;                 // from the keys that can be among a group's largest
      const float least = value.least > kNone ? reach_of(value.least, rz) : INFINITY;
#pragma unroll 1
      for (uint32_t m = in_reach(key, least); m; m &= m - 1) {
        Expert unused;
        t64.add(key64(e0 + __builtin_ctz(m), unused));
      }
      const bool kept64 =
          keep(group_value<double>(t64, lanes, a.group_best, pairs[wave].d, base, base + 16, rz), near);
      kept = sure ? kept64 : kept;
    }
    if (!kept) {
      two = Two<float>();
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = kNone;
    }
  }

  // `cut`: at least top_k keys at or above it, and at most 16 (the lanes) once
  // the error is taken off.  First halving between the two largest keys of
  // every lane alone, whose top_k-th largest is a lower bound of the token's
  // and mostly close to it; then, where that leaves too many, or a token has
  // fewer than top_k such pairs' keys, among all keys.
  const int k = a.top_k;
  float cut = kLowest;
  {
    float lo = fminf(two.best > kNone ? two.best : INFINITY, two.next > kNone ? two.next : INFINITY), hi = two.best;
    lo = row_all(lo, [](float p, float q) { return fminf(p, q); });
    hi = row_all(hi, [](float p, float q) { return fmaxf(p, q); });
    int n = row_count(__ballot(two.best > kNone)) + row_count(__ballot(two.next > kNone));
    const bool enough = n >= k;
    if (enough) cut = lo;
    for (int i = 0; i < 24 && __any(enough && n > k + 1); ++i) {
      const float mid = halfway(lo, hi, i);
      const int m = row_count(__ballot(two.best >= mid)) + row_count(__ballot(two.next >= mid));
      if (m >= k) { lo = mid; n = m; if (enough) cut = mid; }
      else hi = mid;
    }
  }
  auto slack = [&](float c) { return by_logit || c == kLowest ? c : reach_of(c, rz); };
  auto row_total = [&](uint32_t m) {
    return row_all(__builtin_popcount(m), [](int p, int q) { return p + q; });
  };
  uint32_t reach = in_reach(key, slack(cut));
  int n = row_total(reach);
  if (__any(n > 16)) {
    float lo = INFINITY, hi = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      lo = key[v] > kNone ? fminf(lo, key[v]) : lo;
      hi = fmaxf(hi, key[v]);
    }
    lo = row_all(lo, [](float p, float q) { return fminf(p, q); });
    hi = row_all(hi, [](float p, float q) { return fmaxf(p, q); });
    lo = fmaxf(lo, cut);
    for (int i = 0; i < 64 && __any(n > 16); ++i) {
      const float mid = halfway(lo, hi, i);
      if (row_total(in_reach(key, mid)) >= k) {
        lo = mid;
        if (n > 16) {
          reach = in_reach(key, slack(mid));
          n = row_total(reach);
        }
      } else {
        hi = mid;
      }
    }
  }

  int expert = -1, rank = l;
  Expert own = {kNone, 0.0};
  bool chosen = false;
  {
    const bool fits = n <= 16;
    int at = (lane & 48) + row_before(__builtin_popcount(reach));
    if (fits) {
#pragma unroll 1
      for (uint32_t m = reach; m; m &= m - 1) found[wave][at++] = e0 + __builtin_ctz(m);
    }
    wave_sync();
    double k64 = -INFINITY;
    if (fits && l < n) {
      expert = found[wave][lane];
      k64 = key64(expert, own);
    }
    if (!SIGMOID && __any(!sure)) {
      const float k32 = (float)k64;
      const bool close = row_close<15>(k32, 2.0f * key_error(k32, rz)) && !sure && fits && l < n;
      const bool retry = !sure && (n > 16 || row_count(__ballot(close)) > 0);
      if (__any(retry)) {
        const double exact = exact_z();
        z = retry ? exact : z;
        if (retry && fits && l < n) k64 = key64(expert, own);
      }
    }
    // candidates stand in expert order, so equal keys go by lane
    const int r = row_rank<15>(k64);
    if (fits && l < n) {
      rank = r;
      chosen = r < k;
    }
  }
  if (__any(n > 16)) {
    // More experts than lanes within the error of each other (many equal
    // logits): lane j takes the largest (key, expert) that comes after lane
    // j - 1's.  Such a token has top_k of them, as n > 16.
    double last = INFINITY;
    int last_e = -1;
    for (int j = 0; j < k; ++j) {
      double best = -INFINITY;
      int best_e = -1;
      Expert best_x = {0.0f, 0.0};
#pragma unroll 1
      for (int v = 0; v < (kept && n > 16 ? mine : 0); ++v) {
        Expert xv;
        const double q = key64(e0 + v, xv);
        if ((q < last || (q == last && e0 + v > last_e)) && q > best) { best = q; best_e = e0 + v; best_x = xv; }
      }
      const double all = row_all(best, [](double p, double q) { return p > q ? p : q; });
      const int e = row_all(best == all && best_e >= 0 ? best_e : 0x7FFFFFFF, [](int p, int q) { return min(p, q); });
      const uint64_t who = __ballot(best_e == e);
      const int from = __builtin_ctz(((uint32_t)(who >> (lane & 48)) & 0xFFFFu) | 0x10000u) & 15;
      const Expert x = {row_lane(best_x.logit, from), row_lane(best_x.score, from)};
      if (n > 16 && l == j) { expert = e; own = x; chosen = true; }
      last = all;
      last_e = e;
    }
  }
  double s = 0.0;
  if (!SIGMOID && a.renormalize) {
    // the chosen scores up to a common factor, none vanishing
    const float most = row_all(chosen ? own.logit : kNone, [](float p, float q) { return fmaxf(p, q); });
    if (chosen) s = exp((double)own.logit - (double)most);
  } else if (chosen) {
    s = by_logit ? score64(own.logit) : own.score;
  }
  double w = a.scale * s;
  if (a.renormalize) {
    const double sum = row_all(chosen ? s : 0.0, [](double p, double q) { return p + q; });
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (token < a.tokens && (chosen || (l >= n && l < k))) {
    a.index[token * k + rank] = chosen ? expert : -1;
    a.weights[token * k + rank] = chosen ? (float)w : 0.0f;
  }
}

// G lanes a token (16 or 64), experts l * V .. l * V + V - 1 in its lane l, the
// j-th chosen one in lane j.  Chosen experts' gradients are fp64 and meet the
// rest of the row (zeros, or what a softmax takes off) in LDS, from where the
// row goes out in whole vectors.  A softmax's exponentials are fp32, each off
// by a few 2^-24.
template <int DT, int G, int V, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) k_moe_route_bwd(const uint8_t* __restrict__ logits, int64_t tokens, int E,
                                                            int top_k, bool renormalize, double scale,
                                                            const int32_t* __restrict__ index,
                                                            const float* __restrict__ grad_weights,
                                                            uint8_t* __restrict__ grad_logits) {
  __shared__ __attribute__((aligned(16))) float grad[kThreads / G][G * V];
  const int slot = threadIdx.x / G, l = threadIdx.x % G;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / G) + slot;
  const bool on = token < tokens;
  const int64_t at = on ? token * E : 0;
  const uint8_t* row = logits + at * kElemBytes<DT>;
  auto all = [](auto v, auto op) {
    if constexpr (G == 16) return row_all(v, op);
    else return wave_all(v, op);
  };
  auto add = [](double p, double q) { return p + q; };
  const int e0 = l * V;

  int mine = -1;
  double g = 0.0, s = 0.0;
  if (on && l < top_k) {
    mine = index[token * top_k + l];
    if ((unsigned)mine >= (unsigned)E) mine = -1;
    if (mine >= 0) g = (double)grad_weights[token * top_k + l];
  }
  const bool any = all(mine, [](int p, int q) { return max(p, q); }) >= 0;
  float x = -INFINITY;
  if (mine >= 0) x = elem_value<DT>(load_bits<DT>(row + mine * kElemBytes<DT>));
  float out[V];
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = 0.0f;
  float top = 0.0f;
  double z = 1.0;
  if constexpr (!SIGMOID) {
    auto larger = [](float p, float q) { return fmaxf(p, q); };
    if (renormalize) {
      top = all(x, larger);            // a common factor of the scores drops out: the chosen logits are enough
    } else {
      load_logits<DT, V>(row, e0, on && any ? min(V, max(0, E - e0)) : 0, out);
      float most = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) most = fmaxf(most, out[v]);
      top = all(most, larger);
      double sum = 0.0;                // in fp64: next to the largest, 1, the others' sum keeps its own accuracy
#pragma unroll
      for (int v = 0; v < V; ++v) {
        out[v] = out[v] > -INFINITY ? exp_neg(top - out[v]) : 0.0f;
        sum += (double)out[v];
      }
      z = all(sum, add);
    }
  }
  if (mine >= 0) s = SIGMOID ? sigmoid_f64((double)x) : exp((double)x - (double)top) / z;
  double du = scale * g;
  if (renormalize) {
    const double sum = all(s, add), mean = all(g * s, add);
    du = sum > 0.0 ? scale * (g - mean / sum) / sum : 0.0;
  }
  // what a softmax takes off every expert; 0 but for rounding where the weights are renormalized
  const double dot = SIGMOID || renormalize ? 0.0 : all(du * s, add);
  const float off = SIGMOID || renormalize || !any ? 0.0f : (float)(dot / z);
#pragma unroll
  for (int v = 0; v < V; ++v) grad[slot][e0 + v] = SIGMOID || renormalize ? 0.0f : -out[v] * off;
  wave_sync();
  if (mine >= 0) grad[slot][mine] = (float)(SIGMOID ? du * s * (1.0 - s) : s * (du - dot));
  wave_sync();
  if (!on) return;
  // the token's lanes write neighbouring columns together
  uint8_t* to = grad_logits + at * kElemBytes<DT>;
  if (E % 4 == 0) {
#pragma unroll
    for (int v = 0; v < V / 4; ++v) {
      const int e = (v * G + l) * 4;
      if (e >= E) break;
      const float* p = &grad[slot][e];
      if constexpr (DT == DT_F32)
        store16<false>(to + e * 4, u32x4_t{as_u32(p[0]), as_u32(p[1]), as_u32(p[2]), as_u32(p[3])});
      else
        store_8<false>(to + e * 2, u32x2_t{elem_bits<DT>(p[0]) | (elem_bits<DT>(p[1]) << 16),
                                           elem_bits<DT>(p[2]) | (elem_bits<DT>(p[3]) << 16)});
    }
  } else {
    for (int e = l; e < E; e += G) store_bits<DT>(to + e * kElemBytes<DT>, elem_bits<DT>(grad[slot][e]));
  }
}

}  // namespace

// Keys that a lane of k_moe_route_rows is built for, at least n: 0 if there are none.
static int row_width(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 24 ? 24 : n <= 32 ? 32 : 0; }

// The layout of a token's experts in 16 lanes, or one of no lanes.  Runs of a
// whole width, the smallest that holds all experts, where groups are made of
// those (240 experts in 5 groups, 16384 tokens: 11.2 us, and 13.3 with the other);
// otherwise every group gets a power of two of lanes, or its share of the 16 if
// only that holds it, and its experts are dealt out by fours (as they are
// loaded).  Dealt out so, 160 experts in 8 groups take 9.5 us and wave-wide 23.8
// (sigmoid; softmax 12.8 and 28.1), 60 in 4 take 7.6 and with fp64 keys
// throughout 20.9.
static RowLayout row_layout(int experts, int groups, int size) {
  const int v = row_width((experts + 15) / 16);
  int lanes = 16, each = v;
  if (groups > 16 || v == 0) return {0, 0, 0};
  if (groups > 1 && size % v == 0) {
    lanes = size / v;
  } else if (groups > 1) {
    while (lanes * groups > 16) lanes /= 2;
    if (lanes * 32 < size) lanes = 16 / groups;
    each = ((size + lanes - 1) / lanes + 3) / 4 * 4;
    if (row_width(each) == 0) return {0, 0, 0};
  }
  return {lanes, each, 256 / lanes + 1};
}

hipError_t launch_moe_route(const RouteArgs& a, int dt, hipStream_t st) {
  // experts of a lane: enough for 64 lanes, and no group cut inside a lane
  int v = 1;
  while (v * 64 < a.experts) v *= 2;
  const bool whole = a.groups == 1 || (a.experts / a.groups) % v == 0;
  const RowLayout in = row_layout(a.experts, a.groups, a.group_size);
  if (in.lanes > 0 && a.top_k <= 16) {
    const int v16 = row_width(in.each);
    const int64_t grid = (a.tokens + 4 * kTokens - 1) / (4 * kTokens);
    if (!launchable(grid, kThreads)) return hipErrorInvalidValue;
#define LAUNCH(DT, SIGMOID)                                                                    \
  if (v16 == 4) k_moe_route_rows<DT, 4, SIGMOID><<<(unsigned)grid, kThreads, 0, st>>>(a, in);        \
  else if (v16 == 8) k_moe_route_rows<DT, 8, SIGMOID><<<(unsigned)grid, kThreads, 0, st>>>(a, in);   \
  else if (v16 == 16) k_moe_route_rows<DT, 16, SIGMOID><<<(unsigned)grid, kThreads, 0, st>>>(a, in); \
  else if (v16 == 24) k_moe_route_rows<DT, 24, SIGMOID><<<(unsigned)grid, kThreads, 0, st>>>(a, in); \
  else k_moe_route_rows<DT, 32, SIGMOID><<<(unsigned)grid, kThreads, 0, st>>>(a, in)
#define CALL(DT)                            \
  if (a.sigmoid) { LAUNCH(DT, true); }      \
  else { LAUNCH(DT, false); }
    if (dt == DT_F32) { CALL(DT_F32); }
    else if (dt == DT_BF16) { CALL(DT_BF16); }
    else { CALL(DT_F16); }
#undef CALL
#undef LAUNCH
    return hipGetLastError();
  }
  const int64_t blocks = (a.tokens + kTokens - 1) / kTokens;
  if (!launchable(blocks, kThreads)) return hipErrorInvalidValue;
  const size_t lds = (size_t)kTokens * a.experts * sizeof(double);   // at most 32 KB
#define CALL(DT)                                                                             \
  if (!whole) k_moe_route_general<DT><<<(unsigned)blocks, kThreads, lds, st>>>(a);           \
  else if (v == 1) k_moe_route<DT, 1><<<(unsigned)blocks, kThreads, 0, st>>>(a);             \
  else if (v == 2) k_moe_route<DT, 2><<<(unsigned)blocks, kThreads, 0, st>>>(a);             \
  else if (v == 4) k_moe_route<DT, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a);             \
  else if (v == 8) k_moe_route<DT, 8><<<(unsigned)blocks, kThreads, 0, st>>>(a);             \
  else k_moe_route<DT, 16><<<(unsigned)blocks, kThreads, 0, st>>>(a)
  if (dt == DT_F32) { CALL(DT_F32); }
  else if (dt == DT_BF16) { CALL(DT_BF16); }
  else { CALL(DT_F16); }
#undef CALL
  return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void* logits, int dt, int64_t tokens, int experts, int top_k, bool sigmoid,
                                bool renormalize, double scale, const int32_t* index, const float* grad_weights,
                                void* grad_logits, hipStream_t st) {
  const bool rows = experts <= 256 && top_k <= 16;
  const int lanes = rows ? 16 : 64, v = (experts + lanes - 1) / lanes;
  const int64_t blocks = (tokens * lanes + kThreads - 1) / kThreads;
  if (!launchable(blocks, kThreads)) return hipErrorInvalidValue;
#define LAUNCH(DT, G, V, SIGMOID)                                                                             \
  k_moe_route_bwd<DT, G, V, SIGMOID><<<(unsigned)blocks, kThreads, 0, st>>>(                                  \
      (const uint8_t*)logits, tokens, experts, top_k, renormalize, scale, index, grad_weights, (uint8_t*)grad_logits)
#define SIZES(DT, SIGMOID)                                  \
  if (!rows && v <= 8) LAUNCH(DT, 64, 8, SIGMOID);          \
  else if (!rows) LAUNCH(DT, 64, 16, SIGMOID);              \
  else if (v <= 4) LAUNCH(DT, 16, 4, SIGMOID);              \
  else if (v <= 8) LAUNCH(DT, 16, 8, SIGMOID);              \
  else LAUNCH(DT, 16, 16, SIGMOID)
#define CALL(DT)                           \
  if (sigmoid) { SIZES(DT, true); }        \
  else { SIZES(DT, false); }
  if (dt == DT_F32) { CALL(DT_F32); }
  else if (dt == DT_BF16) { CALL(DT_BF16); }
  else { CALL(DT_F16); }
#undef CALL
#undef SIZES
#undef LAUNCH
  return hipGetLastError();
}

}  // namespace mxq
