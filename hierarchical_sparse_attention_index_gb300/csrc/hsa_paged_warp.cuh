// What the warp-MMA kernels of hsa_paged_attn_decode share (paged_attn.cu, paged_four.cu): asynchronous copies, fragments, where a
// piece of 16 keys lies, which keys a row sees, queries in f16, and the merge of the warps and splits.
#pragma once

#include "hsa_paged.cuh"

namespace hsa {

constexpr int kPagedWarps = 4;           // of a CTA
constexpr int kPagedGroup = 16;          // keys of a piece
template <int D>
constexpr int kPagedOutLd = D + 4;       // floats from row to row when the warps merge (bank spread)

__device__ __forceinline__ void page_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, of which all but the first `bytes` are zeros and not read
__device__ __forceinline__ void page_copy16z(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// a row's scales of 4-bit pages, N = 4 or 8 bytes, of which all but the first `bytes` are zeros and not read
template <int N>
__device__ __forceinline__ void page_copy_scales(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void page_copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void page_copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// the 8 x 8 transpose of 16-bit values held two per lane
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    mma_f16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
  }
}

// Where 16 keys from position pos on lie: the piece of the pools in units of 16 rows, times 2^16, plus a bit for each row
// that some query sees; 0 for a bad page or no such row. page_pieces: heads x 16-row pieces of a page; piece_at: where the page,
// number pg of the request, is known to be `page`
template <typename Page>
__device__ __forceinline__ int64_t piece_in(const PagedAttnParams& p, const Span& sp, int b, int h, int64_t page_pieces, int pos, int pg, Page&& page_of) {
  const uint32_t seen = seen32(p, b, sp.lo, sp.hi, sp.gaps, pos) & 0xFFFFu;
  if (!seen) return 0;
  const int page = page_of();
  if (page < 0 || page >= p.n_pages) {
    flag_status(p.status, HSA_FLAG_INDEX_RANGE);
    return 0;
  }
  return ((page * page_pieces + (h * p.page_size + pos - pg * p.page_size) / kPagedGroup) << 16) | seen;
}
__device__ __forceinline__ int64_t piece_at(const PagedAttnParams& p, const Span& sp, int b, int h, int64_t page_pieces, int pos, int pg, int page) {
  return piece_in(p, sp, b, h, page_pieces, pos, pg, [&]() { return page; });
}
__device__ __forceinline__ int64_t find_piece(const PagedAttnParams& p, const Span& sp, int b, int h, int64_t page_pieces, int pos) {
  const int pg = pos / p.page_size;
  return piece_in(p, sp, b, h, page_pieces, pos, pg, [&]() { return p.table[(int64_t)b * p.max_pages + pg]; });
}

// The keys [lo, hi) that a query of length `raw` sees, and those of row r of request b
__device__ __forceinline__ int2 keys_of(const PagedAttnParams& p, int raw, bool flag) {
  const int hi = clamp_vis(p, raw);
  if (raw != hi && flag) flag_status(p.status, HSA_FLAG_INDEX_RANGE);
  return make_int2(p.window > 0 ? max(hi - p.window, 0) : 0, hi);
}
__device__ __forceinline__ int2 row_keys(const PagedAttnParams& p, int b, int r, bool flag) {
  return keys_of(p, p.vis[(int64_t)b * p.nq + r / p.group], flag);
}

// bf16 queries against f16 keys: a thread's elements of a row, which LANES neighbouring lanes hold, to f16, after a power-of-two
// shift of the row, which is taken back in its scale
template <int STEPS, int LANES = 4>
__device__ __forceinline__ void queries_to_f16(uint2 (&x)[STEPS], float& scale) {
  float amax = 0.f;
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks) {
    const uint32_t w[2] = {x[ks].x, x[ks].y};
#pragma unroll
    for (int u = 0; u < 2; ++u)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xFFFF0000u))));
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  int sh = 0;
  if (amax > 0.f && amax < INFINITY) {
    int e;
    frexpf(amax, &e);
    sh = max(-120, min(120, 12 - e));    // amax 2^sh in [2^11, 2^12): products and their sums stay in fp32
  }
  const float mul = __uint_as_float((uint32_t)(127 + sh) << 23);
  scale *= __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks) {
    x[ks].x = pack2<false>(__uint_as_float(x[ks].x << 16) * mul, __uint_as_float(x[ks].x & 0xFFFF0000u) * mul);
    x[ks].y = pack2<false>(__uint_as_float(x[ks].y << 16) * mul, __uint_as_float(x[ks].y & 0xFFFF0000u) * mul);
  }
}

// The warps' parts of rows row0 .. row_end - 1, (m, l) in s_m and s_l and O [row][kPagedOutLd] at `sm`, `stride` bytes from warp to
// warp, become the split's part or, with one split, the result. CLUSTER: the splits of a cluster are joined as well, s_part
// holds this CTA's (m, l).
template <int D, int NT, bool CLUSTER>
__device__ __forceinline__ void merge_warps(const PagedAttnParams& p, const Span& sp, int b, int h, int split, int row0, int row_end, uint8_t* sm,
                                            size_t stride, const float (&s_m)[kPagedWarps][8 * NT], const float (&s_l)[kPagedWarps][8 * NT],
                                            float2* s_part) {
  constexpr int kRows = 8 * NT, kThreads = kPagedWarps * 32, kWarps = kPagedWarps;
  const int tid = threadIdx.x, rows = p.nq * p.group;
  constexpr int kQuads = D / 4;
  auto write_out = [&](int row, int d4, float4 a, float M, float L) {
    const int64_t at = ((int64_t)b * p.nq + row / p.group) * p.heads_q + h * p.group + row % p.group;
    const float inv = L != 0.f ? p.v_scale / L : 0.f;
    uint2 y;
    if (p.q_bf16)
      y = make_uint2(pack2<true>(a.x * inv, a.y * inv), pack2<true>(a.z * inv, a.w * inv));
    else
      y = make_uint2(pack2<false>(a.x * inv, a.y * inv), pack2<false>(a.z * inv, a.w * inv));
    *reinterpret_cast<uint2*>(p.out + at * D + 4 * d4) = y;
    if (p.lse && d4 == 0) p.lse[at] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  };
  // a += 2^(m - M) (O, l); a part in which the row saw no key adds nothing
  auto add = [](float4& a, float& L, float M, float m, float l, float4 x) {
    if (m != -INFINITY || l != 0.f) {
      const float f = m == -INFINITY ? 0.f : ex2_ftz(m - M);
      a.x += f * x.x;
      a.y += f * x.y;
      a.z += f * x.z;
      a.w += f * x.w;
      L += f * l;
    }
  };
  for (int e = tid; e < kRows * kQuads; e += kThreads) {
    const int r = e / kQuads, d4 = e % kQuads, row = row0 + r;
    if (row >= row_end) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    float4* mine = reinterpret_cast<float4*>(sm + ((size_t)r * kPagedOutLd<D> + 4 * d4) * 4);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      add(a, L, M, s_m[w][r], s_l[w][r], *reinterpret_cast<const float4*>(reinterpret_cast<uint8_t*>(mine) + w * stride));
    if (sp.used == 1) {
      if (!CLUSTER || split == 0) write_out(row, d4, a, M, L);
    } else if constexpr (CLUSTER) {
      *mine = a;                         // read by this thread alone until here
      if (d4 == 0) s_part[r] = make_float2(M, L);
    } else {
      const int64_t at = (((int64_t)b * p.heads + h) * p.n_splits + split) * rows + row;
      *reinterpret_cast<float4*>(p.part_o + at * D + 4 * d4) = a;
      if (d4 == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(M, L);
    }
  }
  if constexpr (CLUSTER) {
    if (sp.used == 1) return;            // the same in every CTA of the cluster
    __syncwarp();
    cluster_sync_all();
    // CTA `split` joins every n_splits-th element of the chunk, over the CTAs that have keys
    const uint32_t o_at = smem_u32(sm), ml_at = smem_u32(s_part);
    for (int e = split * kThreads + tid; e < kRows * kQuads; e += p.n_splits * kThreads) {
      const int r = e / kQuads, d4 = e % kQuads, row = row0 + r;
      if (row >= row_end) break;
      float M = -INFINITY;
      for (int c = 0; c < sp.used; ++c) M = fmaxf(M, __uint_as_float((uint32_t)ld_cluster_s32(cluster_map(ml_at + 8 * r, c))));
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll 4
      for (int c = 0; c < sp.used; ++c) {
        const uint64_t ml = ld_cluster_u64(cluster_map(ml_at + 8 * r, c));
        const uint32_t x = cluster_map(o_at + ((uint32_t)r * kPagedOutLd<D> + 4 * d4) * 4, c);
        const uint64_t x0 = ld_cluster_u64(x), x1 = ld_cluster_u64(x + 8);
        float m, l;
        float4 v;
        f2_unpack(ml, m, l);
        f2_unpack(x0, v.x, v.y);
        f2_unpack(x1, v.z, v.w);
        add(a, L, M, m, l, v);
      }
      write_out(row, d4, a, M, L);
    }
    __syncwarp();
    cluster_sync_all();                  // nobody reads this CTA's shared memory any more
  }
}

// A grid of p.n_splits x p.batch x p.heads x p.chunks CTAs. CLUSTER: the splits are one cluster
template <bool CLUSTER, typename Kernel>
cudaError_t launch_splits(Kernel kernel, const PagedAttnParams& p, size_t smem, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_splits * p.batch * p.heads * p.chunks);
  cfg.blockDim = dim3(kPagedWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.n_splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace hsa
