// Keys and values of new tokens into the pages of a dense layer's cache (hsa_paged_cache_write):
//   page[table[b][pos / P]][h][pos % P][:] = round(x[t][h][:] * (1 / scale)),  pos = start[b] + t - cu[b].
//
// A copy with a gather of addresses: it is bound by HBM for prompts and by the chain of dependent
// loads (cu, then start and the table, then the stores) for a single token per request. Measured: 65,536
// tokens (8 heads, 128 dims, bf16) 84.2 us, 6.4 TB/s, to E4M3 73.7; 12,345 tokens (4 heads, 64 dims) to E4M3 6.1 us (4.5
// with the inputs in L2); 64 single tokens 2.7 us. So a block
// issues the loads of its rows first, all of them 16-byte pieces of consecutive threads, looks the
// rows' slots up while they fly (cu in shared memory: one load and a search there instead of a
// chain of global loads), and then stores, 16 bytes per thread along a head's row.
#include "hsa_common.cuh"
#include "hsa_dense.h"
#include "hsa_rows.cuh"

namespace hsa {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kPiecesPerThread = 4;      // 16-byte pieces of K, and as many of V, in flight per thread
constexpr int kBlockPieces = kWriteThreads * kPiecesPerThread;
constexpr int kSpread = 2 * kSms;        // blocks that a copy is spread over before one takes more than it must
constexpr int kCuShared = 1024;          // batches up to this search cu in shared memory

// eight 16-bit values -> eight E4M3 codes of x * inv in fp32 (nearest even, saturating)
__device__ __forceinline__ uint2 to_e4m3x8(uint4 x, float inv, bool bf16) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = half_at(w[i], 0, bf16) * inv, hi = half_at(w[i], 1, bf16) * inv;
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    r[i >> 1] |= (uint32_t)c << (16 * (i & 1));
  }
  return make_uint2(r[0], r[1]);
}

// Request of row t: the b with cu[b] <= t < cu[b + 1], or -1 (padding). `cu` need not be sane:
// the search stays inside [0, batch).
template <typename Cu>
__device__ __forceinline__ int find_request(Cu cu, int batch, int64_t t) {
  int lo = 0, hi = batch;                // the last b of [0, batch) with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return (cu[lo] <= t && t < cu[lo + 1]) ? lo : -1;
}

// E4M3: 16 input elements (two loads) make one 16-byte piece; else 8 elements, one load
template <bool E4M3>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  __shared__ int32_t s_cu[kCuShared + 1];
  __shared__ int64_t s_slot[kBlockPieces];   // per row of the block: (page * heads) * P + pos % P, or -1
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kElems = E4M3 ? 16 : 8, kLoads = E4M3 ? 2 : 1;
  const int ppr = p.heads * p.head_dim / kElems;         // pieces per row
  const int rows = p.rows_per_block;
  const int64_t t0 = (int64_t)blockIdx.x * rows;
  const int n_rows = (int)imin64(rows, p.n_tokens - t0);
  const int tid = threadIdx.x;
  const int pieces = n_rows * ppr;
  const int pph = p.head_dim / kElems;                   // pieces per head
  for (int base = 0; base < pieces; base += kBlockPieces) {
    uint4 x[2][kPiecesPerThread][kLoads];
#pragma unroll
    for (int i = 0; i < kPiecesPerThread; ++i) {
      const int e = base + i * kWriteThreads + tid;
      if (e < pieces) {
        const int r = e / ppr, c = e - r * ppr;
        const uint4* k = reinterpret_cast<const uint4*>(p.k + (t0 + r) * p.k_stride + (int64_t)c * kElems);
        const uint4* v = reinterpret_cast<const uint4*>(p.v + (t0 + r) * p.v_stride + (int64_t)c * kElems);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          x[0][i][u] = __ldcs(k + u);
          x[1][i][u] = __ldcs(v + u);
        }
      }
    }
    if (base == 0) {
      const bool shared = p.cu && p.batch <= kCuShared;
      if (shared)
        for (int i = tid; i <= p.batch; i += kWriteThreads) s_cu[i] = p.cu[i];
      __syncthreads();
      for (int r = tid; r < n_rows; r += kWriteThreads) {
        const int64_t t = t0 + r;
        int b;
        int64_t first;
        if (!p.cu) {
          b = (int)(t / p.per_request);
          first = (int64_t)b * p.per_request;
        } else {
          b = shared ? find_request(s_cu, p.batch, t) : find_request(p.cu, p.batch, t);
          first = b < 0 ? 0 : (shared ? s_cu[b] : p.cu[b]);
        }
        int64_t slot = -1;
        if (b >= 0) {
          const int64_t pos = (p.start ? p.start[b] : 0) + (t - first);
          const int64_t pg = pos >= 0 ? pos / p.page_size : p.max_pages;
          if (pg < p.max_pages) {
            const int64_t page = p.table[(int64_t)b * p.max_pages + pg];
            if (page >= 0 && page < p.n_pages) slot = page * p.heads * p.page_size + pos % p.page_size;
          }
          if (slot < 0) flag_status(p.status, HSA_FLAG_WRITE_RANGE);
        }
        s_slot[r] = slot;
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kPiecesPerThread; ++i) {
      const int e = base + i * kWriteThreads + tid;
      if (e < pieces) {
        const int r = e / ppr, c = e - r * ppr;
        const int64_t slot = s_slot[r];
        if (slot >= 0) {
          const int h = c / pph, ch = c - h * pph;
          const int64_t at = (slot + (int64_t)h * p.page_size) * pph + ch;   // in 16-byte pieces
          uint4* pool[2] = {reinterpret_cast<uint4*>(p.k_pool), reinterpret_cast<uint4*>(p.v_pool)};
          const float inv[2] = {p.k_inv, p.v_inv};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint4 y = x[s][i][0];
            if constexpr (E4M3) {
              const uint2 a = to_e4m3x8(x[s][i][0], inv[s], p.bf16), b2 = to_e4m3x8(x[s][i][kLoads - 1], inv[s], p.bf16);
              y = make_uint4(a.x, a.y, b2.x, b2.y);
            }
            pool[s][at] = y;
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteParams& p0, bool e4m3, cudaStream_t s) {
  PagedWriteParams p = p0;
  const int ppr = p.heads * p.head_dim / (e4m3 ? 16 : 8);
  // whole rows: up to kBlockPieces pieces a block (a row of more pieces is copied in turns), and fewer,
  // down to one piece per thread, while there are SMs without a block
  const int64_t most = imax64(1, kBlockPieces / ppr), least = imax64(1, kWriteThreads / ppr);
  p.rows_per_block = (int32_t)imin64(most, imax64(least, (p.n_tokens + kSpread - 1) / kSpread));
  const int64_t blocks = (p.n_tokens + p.rows_per_block - 1) / p.rows_per_block;
  auto kernel = e4m3 ? paged_write_kernel<true> : paged_write_kernel<false>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kWriteThreads), 0, s, p);
}

}  // namespace hsa
