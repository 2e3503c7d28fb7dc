// Host-side declarations of the dense attention calls: parameter blocks, how the work is cut, launchers.
// Not part of the public ABI.
#pragma once

#include "hsa_internal.h"

namespace hsa {

constexpr int kSms = 152;                // of a GB300; rules that also answer without a device go by it

// ------------------------------------------------------------------ dense attention over a paged cache
struct PagedWriteParams {
  int32_t batch, heads, head_dim, page_size;
  int64_t n_pages, max_pages;
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int32_t* table;
  float k_inv, v_inv;     // fp32 reciprocals of the scales
  const uint16_t* k;      // [n_tokens][heads][head_dim], k_stride elements from row to row
  const uint16_t* v;
  int64_t k_stride, v_stride, n_tokens;
  int32_t bf16;           // 1: k and v are bf16, 0: f16
  int32_t rows_per_block; // set by the launcher
  const int32_t* cu;      // [batch + 1] or NULL: per_request rows each
  int64_t per_request;
  const int64_t* start;   // [batch] or NULL
  uint32_t* status;
};
cudaError_t launch_paged_write(const PagedWriteParams& p, bool e4m3, cudaStream_t s);

// How hsa_paged_attn_decode cuts its work (host only; the workspace holds n_splits partials per
// row where a join follows)
struct PagedSplit {
  bool tc;                // paged_rows_kernel (tcgen05), else paged_attn_kernel
  int32_t chunk_rows;     // query rows (queries x heads of a group) per CTA
  int32_t chunks;         // CTAs that share a key-value head's rows
  int32_t n_splits;       // CTAs along the cache's length
  int32_t split_len;      // keys per split, at least
  int32_t align;          // splits start at multiples of this
  bool cluster;           // the splits are one thread-block cluster, which joins them
  bool joined;            // paged_join_kernel follows
};
PagedSplit paged_split(int32_t batch, int32_t heads, int32_t group, int32_t nq, int64_t max_vis, int32_t window, int32_t kv_dtype);
int64_t paged_splits_most(int32_t batch, int32_t heads, int32_t group, int32_t nq, int64_t max_vis, int32_t kv_dtype);

struct PagedAttnParams {
  int32_t batch, heads, page_size;
  int64_t n_pages, max_pages;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  const uint16_t* q;      // [B][nq][heads_q][D]
  int32_t q_bf16;         // q and out are bf16, else f16
  int32_t heads_q, group, nq, window;
  const int32_t* vis;     // [B][nq]
  int64_t max_vis;
  float scale_log2;       // sm_scale * k_scale * log2 e
  float v_scale;
  int32_t chunk_rows, chunks, n_splits, split_len, align, cluster;   // PagedSplit
  uint16_t* out;
  float* lse;             // or NULL
  float* part_o;          // workspace [B][heads][n_splits][rows][D], unnormalised
  float* part_ml;         // workspace [B][heads][n_splits][rows] (log2 of the unit of the sums, sum)
  uint32_t* status;
};
cudaError_t launch_paged_attn(const PagedAttnParams& p, const PagedSplit& sp, int32_t head_dim, int32_t kv_dtype, uint64_t wait_ns,
                              cudaStream_t s);
cudaError_t launch_paged_rows(const PagedAttnParams& p, int32_t head_dim, int32_t kv_dtype, uint64_t wait_ns, cudaStream_t s);

// The driver's tensor-map encoder, looked up once through the runtime (no libcuda link); NULL: none.
using TensorMapEncoder = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncoder tensor_map_encoder();

// ------------------------------------------------------------------ causal attention over packed prompts
int64_t prompt_blocks(const hsa_prompt_args& a);
cudaError_t launch_prompt_attn(const hsa_prompt_args& a, uint32_t* status, uint64_t wait_ns, cudaStream_t s);

}  // namespace hsa
