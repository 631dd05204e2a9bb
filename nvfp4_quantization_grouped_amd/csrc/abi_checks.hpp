// Host-side checks that the C ABI's parts share: which buffers overlap, types,
// alignment, products of sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq.h"

namespace mxq {

// A buffer of a call: where it starts and how many bytes it holds.
struct Span {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && pa < pb + (uintptr_t)b.bytes && pb < pa + (uintptr_t)a.bytes;
}
// Does the output `out` overlap any of the `n` others?
inline bool overlaps_any(const Span& out, const Span* others, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(out, others[i])) return true;
  return false;
}

inline bool dtype_ok(int t) { return t == MXQ_F32 || t == MXQ_BF16 || t == MXQ_F16; }
inline int64_t dtype_bytes(int t) { return t == MXQ_F32 ? 4 : 2; }
inline bool misaligned4(const void* p) { return ((uintptr_t)p & 3) != 0; }
inline int from_hip(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

// a * b for a, b >= 0, or -1 when it reaches `limit`.
inline int64_t product_below(int64_t a, int64_t b, int64_t limit) {
  if (a == 0 || b == 0) return 0;
  return a > (limit - 1) / b ? -1 : a * b;
}

}  // namespace mxq
