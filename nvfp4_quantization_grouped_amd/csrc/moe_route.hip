// The router: scores, balance bias, expert groups, top-k and weights
// (moe_route), and the weights' gradient with respect to the logits.
//
// One wave per token.  The keys that decide the choice are fp64: two experts
// whose scores differ by less than fp32 resolves are still told apart, and
// equal ones go to the lower index.  Each wave holds its token's keys in LDS;
// a chosen expert's key is overwritten with -inf.
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
  double s = 0.0;
  if (mine >= 0) s = score(elem_value<DT>(load_bits<DT>(x + mine * kElemBytes<DT>)));
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
__global__ void __launch_bounds__(kThreads) k_moe_route(RouteArgs a) {
  extern __shared__ double keys[];
  const int wave = threadIdx.x >> 6;
  const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
  if (token < a.tokens) route_token<DT>(a, token, keys + wave * a.experts);
}

// One wave per token; u: experts floats of the wave's own LDS, the gradient of each score.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_moe_route_bwd(const uint8_t* __restrict__ logits, int64_t tokens, int E,
                                                            int top_k, bool sigmoid, bool renormalize, double scale,
                                                            const int32_t* __restrict__ index,
                                                            const float* __restrict__ grad_weights,
                                                            uint8_t* __restrict__ grad_logits) {
  extern __shared__ float rows_u[];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
  if (token >= tokens) return;
  float* u = rows_u + wave * E;
  const uint8_t* x = logits + token * E * kElemBytes<DT>;
  uint8_t* out = grad_logits + token * E * kElemBytes<DT>;
  int mine = -1;
  double g = 0.0;
  if (lane < top_k) {
    mine = index[token * top_k + lane];
    if ((unsigned)mine >= (unsigned)E) mine = -1;
    if (mine >= 0) g = (double)grad_weights[token * top_k + lane];
  }
  const bool any = __ballot(mine >= 0) != 0;
  float top = -INFINITY;
  double z = 1.0;
  if (!sigmoid && any) {
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
  double s = 0.0;
  if (mine >= 0) {
    const double v = (double)elem_value<DT>(load_bits<DT>(x + mine * kElemBytes<DT>));
    s = sigmoid ? sigmoid_f64(v) : exp(v - (double)top) / z;
  }
  double du = scale * g;
  if (renormalize) {
    const double sum = wave_sum(s), mean = wave_sum(g * s);
    du = sum > 0.0 ? scale * (g - mean / sum) / sum : 0.0;
  }
  const double dot = sigmoid || !any ? 0.0 : wave_sum(mine >= 0 ? du * s : 0.0);
  for (int e = lane; e < E; e += 64) {
    float v = 0.0f;
    if (!sigmoid && any) {
      const float l = elem_value<DT>(load_bits<DT>(x + e * kElemBytes<DT>));
      // what the sum of all gradients takes off; with renormalized weights it is 0 but for rounding
      if (eligible(l) && !renormalize) v = (float)(-exp((double)l - (double)top) / z * dot);
    }
    u[e] = v;
  }
  wave_sync();
  if (mine >= 0) u[mine] = (float)(sigmoid ? du * s * (1.0 - s) : renormalize ? du * s : s * (du - dot));
  wave_sync();
  for (int e = lane; e < E; e += 64) store_bits<DT>(out + e * kElemBytes<DT>, elem_bits<DT>(u[e]));
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, int dt, hipStream_t st) {
  const int64_t blocks = (a.tokens + kTokens - 1) / kTokens;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const size_t lds = (size_t)kTokens * a.experts * sizeof(double);   // at most 32 KB
  if (dt == DT_F32) k_moe_route<DT_F32><<<(unsigned)blocks, kThreads, lds, st>>>(a);
  else if (dt == DT_BF16) k_moe_route<DT_BF16><<<(unsigned)blocks, kThreads, lds, st>>>(a);
  else k_moe_route<DT_F16><<<(unsigned)blocks, kThreads, lds, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void* logits, int dt, int64_t tokens, int experts, int top_k, bool sigmoid,
                                bool renormalize, double scale, const int32_t* index, const float* grad_weights,
                                void* grad_logits, hipStream_t st) {
  const int64_t blocks = (tokens + kTokens - 1) / kTokens;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const size_t lds = (size_t)kTokens * experts * sizeof(float);
#define CALL(DT)                                                                                                  \
  k_moe_route_bwd<DT><<<(unsigned)blocks, kThreads, lds, st>>>((const uint8_t*)logits, tokens, experts, top_k,    \
                                                               sigmoid, renormalize, scale, index, grad_weights, \
                                                               (uint8_t*)grad_logits)
  if (dt == DT_F32) CALL(DT_F32);
  else if (dt == DT_BF16) CALL(DT_BF16);
  else CALL(DT_F16);
#undef CALL
  return hipGetLastError();
}

}  // namespace mxq
