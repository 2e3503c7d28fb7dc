// What the kernels of hsa_paged_attn_decode share: the positions that the queries of a request see,
// cut into splits.
#pragma once

#include "hsa_common.cuh"
#include "hsa_dense.h"

namespace hsa {

// The positions some query of request b sees, [lo, hi), and each split's share of them
struct Span {
  int lo, hi, base, len, used;           // split s: [base + s len, base + (s + 1) len) cut to hi; `used` of them hold any
};
__device__ __forceinline__ int clamp_vis(const PagedAttnParams& p, int v) { return min(max(v, 0), (int)p.max_vis); }
__device__ __forceinline__ Span request_span(const PagedAttnParams& p, int b) {
  Span s;
  s.lo = 0x7fffffff;
  s.hi = 0;
  static_assert(HSA_MAX_NQ <= 8, "one turn of loads");
  const int32_t* vis = p.vis + (int64_t)b * p.nq;
  int v[HSA_MAX_NQ];                     // loaded together: one after the other they would hold up the start
#pragma unroll
  for (int i = 0; i < HSA_MAX_NQ; ++i) v[i] = i < p.nq ? vis[i] : 0;
#pragma unroll
  for (int i = 0; i < HSA_MAX_NQ; ++i) {
    const int x = clamp_vis(p, v[i]);
    s.hi = max(s.hi, x);
    if (x > 0) s.lo = min(s.lo, p.window > 0 ? max(x - p.window, 0) : 0);
  }
  if (s.hi == 0) s.lo = 0;
  s.base = s.lo & ~(p.align - 1);
  const int need = (s.hi - s.base + p.n_splits - 1) / p.n_splits;
  s.len = max(p.split_len, (need + 63) & ~63);
  s.used = max(1, (s.hi - s.base + s.len - 1) / s.len);
  return s;
}

}  // namespace hsa
