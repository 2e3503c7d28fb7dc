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
  for (int i = 0; i < p.nq; ++i) {
    const int v = clamp_vis(p, p.vis[(int64_t)b * p.nq + i]);
    s.hi = max(s.hi, v);
    if (v > 0) s.lo = min(s.lo, p.window > 0 ? max(v - p.window, 0) : 0);
  }
  if (s.hi == 0) s.lo = 0;
  s.base = s.lo & ~(p.align - 1);
  const int need = (s.hi - s.base + p.n_splits - 1) / p.n_splits;
  s.len = max(p.split_len, (need + 63) & ~63);
  s.used = max(1, (s.hi - s.base + s.len - 1) / s.len);
  return s;
}

}  // namespace hsa
