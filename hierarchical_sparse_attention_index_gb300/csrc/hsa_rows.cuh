// What the kernels between rows of tokens and pages share: the request, position and slot of each row of a block.
#pragma once

#include "hsa_common.cuh"
#include "hsa_dense.h"

namespace hsa {

constexpr int kSlotRows = 32;            // rows of a block at most
constexpr int kSlotCu = 1024;            // batches up to this search cu in shared memory

struct RowSlots {
  int32_t cu[kSlotCu + 1];
  int64_t pos[kSlotRows];                // position of row r in its request; 0 for padding
  int64_t slot[kSlotRows];               // (page * heads) * P + pos % P, or -1: padding or no such place
  bool real[kSlotRows];                  // not padding
};

__device__ __forceinline__ float half_at(uint32_t w, int hi, bool bf16) {
  if (bf16) return __uint_as_float(hi ? (w & 0xFFFF0000u) : (w << 16));
  return __half2float(__ushort_as_half((unsigned short)(hi ? (w >> 16) : (w & 0xFFFFu))));
}

// Fills s for rows t0 .. t0 + n_rows - 1; a row without a place in the pool sets `flag`. Every thread of the block calls
// it; what it wrote can be read after it. `cu` need not be sane: the search stays inside [0, batch).
__device__ __forceinline__ void find_slots(const PagedWriteParams& p, int64_t t0, int n_rows, RowSlots& s, uint32_t flag) {
  const bool shared = p.cu && p.batch <= kSlotCu;
  if (shared)
    for (int i = threadIdx.x; i <= p.batch; i += blockDim.x) s.cu[i] = p.cu[i];
  __syncthreads();
  const int r = threadIdx.x;
  if (r < n_rows) {
    const int64_t t = t0 + r;
    const int32_t* cu = shared ? s.cu : p.cu;
    int b;
    int64_t first;
    bool real = true;
    if (!cu) {
      b = (int)(t / p.per_request);
      first = (int64_t)b * p.per_request;
    } else {
      int lo = 0, hi = p.batch;          // the last b of [0, batch) with cu[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
      }
      b = lo;
      first = cu[b];
      real = first <= t && t < cu[b + 1];
    }
    int64_t pos = 0, slot = -1;
    if (real) {
      pos = (p.start ? p.start[b] : 0) + (t - first);
      const int64_t pg = pos >= 0 ? pos / p.page_size : p.max_pages;
      if (pg < p.max_pages) {
        const int64_t page = p.table[(int64_t)b * p.max_pages + pg];
        if (page >= 0 && page < p.n_pages) slot = page * p.heads * p.page_size + pos % p.page_size;
      }
      if (slot < 0 && flag) flag_status(p.status, flag);
    }
    s.pos[r] = pos;
    s.slot[r] = slot;
    s.real[r] = real;
  }
  __syncthreads();
}

}  // namespace hsa
