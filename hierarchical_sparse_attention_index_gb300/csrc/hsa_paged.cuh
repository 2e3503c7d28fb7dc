// What the kernels of hsa_paged_attn_decode share: the positions that the queries of a request see,
// cut into splits.
#pragma once

#include "hsa_common.cuh"
#include "hsa_dense.h"
#include "hsa_softmax.cuh"

namespace hsa {

// The positions some query of request b sees lie in [lo, hi); each split's share of that
struct Span {
  int lo, hi, base, len, used;           // split s: [base + s len, base + (s + 1) len) cut to hi; `used` of them hold any
  bool gaps;                             // queries further apart than the window: some of [lo, hi) may be seen by none
};
__device__ __forceinline__ int clamp_vis(const PagedAttnParams& p, int v) { return min(max(v, 0), (int)p.max_vis); }
__device__ __forceinline__ Span request_span(const PagedAttnParams& p, int b) {
  Span s;
  int least = 0x7fffffff;                // the shortest length that is not 0
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
    if (x > 0) least = min(least, x);
  }
  s.lo = p.window > 0 && s.hi > 0 ? max(least - p.window, 0) : 0;
  s.gaps = p.window > 0 && s.hi - p.window > least;
  s.base = s.lo & ~(p.align - 1);
  const int need = (s.hi - s.base + p.n_splits - 1) / p.n_splits;
  s.len = max(p.split_len, (need + 63) & ~63);
  s.used = max(1, (s.hi - s.base + s.len - 1) / s.len);
  return s;
}
// Bits [lo, hi) of a word, either border cut to 0 .. 32
__device__ __forceinline__ uint32_t bits32(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? 0xFFFFFFFFu : (1u << max(hi, 0)) - 1u, below_lo = lo >= 32 ? 0xFFFFFFFFu : (1u << max(lo, 0)) - 1u;
  return below_hi & ~below_lo;
}
// Bit i: some query of request b, whose Span has lo, hi and gaps, sees position at + i
__device__ __forceinline__ uint32_t seen32(const PagedAttnParams& p, int b, int lo, int hi, bool gaps, int at) {
  if (__builtin_expect(!gaps, 1)) return bits32(lo - at, hi - at);
  uint32_t seen = 0;
#pragma unroll 1
  for (int i = 0; i < p.nq; ++i) {
    const int x = clamp_vis(p, p.vis[(int64_t)b * p.nq + i]);
    seen |= bits32(max(x - p.window, 0) - at, x - at);
  }
  return seen;
}

}  // namespace hsa
