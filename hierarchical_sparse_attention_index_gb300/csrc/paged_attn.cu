// Attention of a few new tokens per request over a paged key-value cache (hsa_paged_attn_decode):
//   o = sum_j softmax_j(scale q.k_j) v_j over the positions j a query sees, split over the
// cache's length and joined.
//
// Bound: every key and value is read once and used by nq x group query rows only, so the reads
// from HBM decide, and beside them the instructions that a warp spends on a key. Hence
//  - one CTA per (request, key-value head, up to 32 query rows, split of the length); the rows are
//    the queries and the heads of the group together, so that grouped heads share every load;
//  - inside a CTA each of 4 warps streams its own 16-key groups (a group never leaves a page)
//    through a private ring of cp.async stages: 16 rows of one head lie in one contiguous piece, no
//    block barrier is ever needed, and two or three CTAs per SM keep up to 192 KB in flight;
//  - products by the warp MMA m16n8k16, transposed: S^T = K Q^T and O^T += V^T P^T, so that keys and
//    dims fill the 16-row side and queries the 8-column side. Most calls have 8 rows or fewer; with
//    the queries on the 16-row side half of every product, exponential and accumulator would be
//    padding. (A tcgen05 instruction takes 128 rows.) The k index is permuted so that a thread's
//    fragments of K are the 16-byte pieces of its rows: one shared load feeds two (16-bit) or four
//    (E4M3) k-steps. V goes through transposed matrix loads, or, in E4M3, byte permutes and converts
//    in registers; P^T comes from S^T's accumulators by movmatrix;
//  - softmax in one pass with the running maximum and sum in fp32. The maximum is only raised, and
//    the outputs rescaled, when some logit passes it by 2^8, and most groups need one vote instead of shuffles. The
//    weights then stay below 2^8, which bf16 holds; in f16 they are 2^7 times that, as its full steps end at 2^-14;
//  - the weights P are rounded to the 16-bit operand type of the product with V (off by at most a relative 2^-8 in
//    bf16, in f16 2^-11 down to 2^-21 of a row's largest weight and 2^-32 of it below, independent from key to key); the
//    sum l takes them unrounded.
// The four warps' (m, l, O) are merged in shared memory. With one split the CTA writes the result. Up to
// 8 splits are one thread-block cluster, whose CTAs join their parts through distributed shared memory;
// more leave their parts in the workspace, and paged_join_kernel joins them. Either joins in order.
#include "hsa_paged.cuh"

namespace hsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;               // keys per stage of a warp
constexpr int32_t kTcRows = 24;          // 16-bit pages: more query rows than this take the tcgen05 kernel

enum KvType { kBf16 = HSA_BF16, kF16 = HSA_F16, kE4M3 = HSA_E4M3, kE2M1 = HSA_E2M1 };

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, of which all but the first `bytes` are zeros and not read
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// a row's scales of 4-bit pages, N = 4 or 8 bytes, of which all but the first `bytes` are zeros and not read
template <int N>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
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
// 4-bit pages: the key of a 16-key group at place i of the products' key index, and back. Thread t's keys, places
// 2t, 2t + 1, 2t + 8 and 2t + 9, are then t, t + 4, t + 8, t + 12
__host__ __device__ __forceinline__ constexpr int four_key(int i) { return (i & 8) + ((i & 1) << 2) + ((i & 6) >> 1); }
__host__ __device__ __forceinline__ constexpr int four_place(int r) { return (r & 8) + ((r & 3) << 1) + ((r & 4) >> 2); }
// (x, x) of the low or the high half of an f16 pair times y
__device__ __forceinline__ uint32_t mul_half(uint32_t x, int hi, uint32_t y) {
  const __half2 a = *reinterpret_cast<const __half2*>(&x), b = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hmul2(hi ? __high2half2(a) : __low2half2(a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_pair(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// CTAs that an SM holds, for NT tiles of 8 query rows: as registers and shared memory (their rings, 227 KB) allow
constexpr int ctas_per_sm(int nt) { return nt <= 2 ? 3 : 2; }

template <int D, int KV, int NT>
struct Tile {
  static constexpr int kElem = KV == kE4M3 ? 1 : 2;
  static constexpr int kRow = KV == kE2M1 ? D / 2 : D * kElem;           // bytes of a key's row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kHalf = kGroup * kRow;            // K, then V
  static constexpr int kScaleRow = KV == kE2M1 ? D / 16 : 0;             // bytes of a row's scales
  static constexpr int kScales = kGroup * kScaleRow;     // K's behind V, then V's
  static constexpr int kStage = 2 * kHalf + 2 * kScales;
  static constexpr int kCtas = ctas_per_sm(NT);
  static constexpr int kRingMax = kCtas == 3 ? 16384 : 24576;
  static constexpr int kStagesMax = KV == kE2M1 ? (D == 128 ? 10 : 15) : 6;
  static constexpr int kStages = kRingMax / kStage > kStagesMax ? kStagesMax : kRingMax / kStage;
  static constexpr int kRing = kStage * kStages;
  static constexpr int kOutLd = D + 4;                   // floats from row to row when the warps merge (bank spread)
  static_assert(8 * NT * kOutLd * 4 <= kRing, "a warp's outputs fit its ring");
  // 16-byte piece c of row r. K: pieces 4i..4i+3 of two neighbouring rows are read together; V: one
  // piece of 8 rows (matrix loads), or two pieces of rows 0, 2, 4, 6 (E4M3)
  // E2M1: K's row r lies at its place in the products (four_key(place) = r), so that 8 lanes read 128 bytes in a row; V's pieces
  // of rows t and 4 + t are read together by thread t, 8 (4) bytes of each by 8 threads
  static __device__ __forceinline__ uint32_t k_at(int r, int c) {
    if constexpr (KV == kE2M1) return (uint32_t)(four_place(r) * kRow + c * 16);
    return (uint32_t)(r * kRow + (kChunks >= 8 ? (c ^ ((r & 1) << 2)) : c) * 16);
  }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) {
    if constexpr (KV == kE2M1) return (uint32_t)(r * kRow + (kChunks == 4 ? c ^ (r & 2) : c) * 16);
    return (uint32_t)(r * kRow + (kChunks >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) * 16);
  }
};

// NT: tiles of 8 query rows
// CLUSTER: the splits of a (request, head, chunk) are one cluster
template <int D, int KV, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, (Tile<D, KV, NT>::kCtas)) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  using T = Tile<D, KV, NT>;
  constexpr bool kB = KV == kBf16;                       // products in bf16, else in f16
  constexpr float lift = kLift<kB>;                      // weights are 2^(x - m), m that much below the running maximum
  constexpr int kSteps = D / 16, kMt = D / 16, kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_scale[kRows];
  __shared__ int s_lo[kRows], s_hi[kRows];
  __shared__ float2 s_part[kRows];                       // CLUSTER: (m, l) of this CTA's part of each row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  griddep_wait();
  griddep_launch_dependents();

  int idx = blockIdx.x, split = 0;
  if constexpr (CLUSTER) {
    split = idx % p.n_splits;
    idx /= p.n_splits;
  }
  const int chunk = idx % p.chunks;
  idx /= p.chunks;
  const int h = idx % p.heads;
  idx /= p.heads;
  const int b = idx % p.batch;
  if constexpr (!CLUSTER) split = idx / p.batch;
  const Span sp = request_span(p, b);
  if (!CLUSTER && split >= sp.used) return;
  const int begin = sp.base + split * sp.len, end = max(begin, min(begin + sp.len, sp.hi));   // keys of this CTA
  const int rows = p.nq * p.group, row0 = chunk * p.chunk_rows, row_end = min(row0 + p.chunk_rows, rows);

  // ---------------------------------------------------------------- the ring: 16-key groups of this warp
  const uint32_t ring = smem_u32(sm) + (uint32_t)warp * T::kRing;
  const int n_groups = max(0, (end - begin + kGroup * (kWarps - warp) - 1) / (kGroup * kWarps));
  uint32_t bad = 0;                                      // bit s: the group in stage s is not loaded
  // where 32 groups lie, one per lane, looked up a turn ahead of their use: the piece of the pools in
  // units of 16 rows, times 2^16, plus a bit for each row that some query sees; 0 for a bad page or no such row
  const int64_t page_pieces = (int64_t)p.heads * (p.page_size / kGroup);
  auto find_pieces = [&](int turn) -> int64_t {
    const int i = 32 * turn + lane;
    if (i >= n_groups) return 0;
    const int pos = begin + kGroup * (warp + kWarps * i), pg = pos / p.page_size;
    const uint32_t seen = seen32(p, b, sp.lo, sp.hi, sp.gaps, pos) & 0xFFFFu;
    if (!seen) return 0;
    const int page = p.table[(int64_t)b * p.max_pages + pg];
    if (page < 0 || page >= p.n_pages) {
      flag_status(p.status, HSA_FLAG_INDEX_RANGE);
      return 0;
    }
    return ((page * page_pieces + (h * p.page_size + pos - pg * p.page_size) / kGroup) << 16) | seen;
  };
  int64_t pieces = find_pieces(0), pieces_next = find_pieces(1);
  auto issue = [&](int i, int stage) {                   // called with i = 0, 1, 2, ...
    const int64_t found = __shfl_sync(0xffffffffu, pieces, i & 31);
    if ((i & 31) == 31) {
      pieces = pieces_next;
      pieces_next = find_pieces((i >> 5) + 2);
    }
    if (i < n_groups) {
      const uint32_t st = (uint32_t)stage * T::kStage, seen = (uint32_t)found & 0xFFFFu;
      if constexpr (KV == kE2M1) {
        // a lane for each row's scales: of K where it lies among the keys, of V in the order t, t + 4, .. of thread t
        const int r = lane & 15;
        const uint32_t n = (seen >> r) & 1u ? (uint32_t)T::kScaleRow : 0u;
        const uint8_t* src = (lane < 16 ? p.k_s : p.v_s) + (n ? ((found >> 16) * kGroup + r) * T::kScaleRow : 0);
        const uint32_t place = lane < 16 ? four_place(r) : kGroup + (r & 3) * 4 + (r >> 2);
        cp_async_scales<(T::kScaleRow ? T::kScaleRow : 4)>(ring + st + 2 * T::kHalf + place * T::kScaleRow, src, n);
      }
      bad = (bad & ~(1u << stage)) | ((seen ? 0u : 1u) << stage);
      const int64_t at = seen ? (found >> 16) * (kGroup * T::kRow) + lane * 16 : 0;
      const uint8_t* k = p.k_pool + at;
      const uint8_t* v = p.v_pool + at;
      constexpr int kCopies = kGroup * T::kChunks / 32;
      if (seen == 0xFFFFu) {
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          cp_async16(ring + T::k_at((u * 32 + lane) / T::kChunks, lane % T::kChunks) + st, k + u * 512);
          cp_async16(ring + T::kHalf + T::v_at((u * 32 + lane) / T::kChunks, lane % T::kChunks) + st, v + u * 512);
        }
      } else {
        // rows no query sees are not read: they become zeros, whatever the pool holds there
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          const int r = (u * 32 + lane) / T::kChunks;
          const uint32_t n = (seen >> r) & 1u ? 16u : 0u;
          cp_async16z(ring + T::k_at((u * 32 + lane) / T::kChunks, lane % T::kChunks) + st, k + (n ? u * 512 : 0), n);
          cp_async16z(ring + T::kHalf + T::v_at((u * 32 + lane) / T::kChunks, lane % T::kChunks) + st, v + (n ? u * 512 : 0), n);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < T::kStages - 1; ++s) issue(s, s);

  // ---------------------------------------------------------------- each row's keys, for masked groups
  int all_lo = 0, all_hi = 0x7fffffff;                   // inside [all_lo, all_hi) no row masks anything
  if (lane < kRows) {
    const int r = row0 + lane;
    int lo = 0, hi = 0;
    if (r < row_end) {
      const int raw = p.vis[(int64_t)b * p.nq + r / p.group];
      hi = clamp_vis(p, raw);
      if (raw != hi && split == 0 && h == 0) flag_status(p.status, HSA_FLAG_INDEX_RANGE);
      lo = p.window > 0 ? max(hi - p.window, 0) : 0;
      all_lo = lo;
      all_hi = hi;
    }
    if (warp == 0) {
      s_lo[lane] = lo;
      s_hi[lane] = hi;
    }
  }
  all_lo = __reduce_max_sync(0xffffffffu, all_lo);
  all_hi = __reduce_min_sync(0xffffffffu, all_hi);

  // ---------------------------------------------------------------- queries into B fragments
  // k-step ks covers, of thread t, the 4 consecutive elements that its piece of a key's row brings
  // to that step
  uint32_t qb[NT][kSteps][2];
  constexpr bool kScaled = KV == kE4M3 || KV == kE2M1;
  constexpr int kScales = kScaled ? 2 * NT : 1;
  float scale[kScales];                                  // of rows 2t, 2t + 1 of each tile (or of all rows)
  {
    constexpr int kPer = KV == kE2M1 ? 4 : 16 / T::kElem;                // consecutive elements of a thread: of a 16-byte piece, 4 of a scale's group
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool real = r < row_end;
      const int qi = real ? r / p.group : 0, hq = h * p.group + (real ? r % p.group : 0);
      const uint16_t* q = p.q + (((int64_t)b * p.nq + qi) * p.heads_q + hq) * D;
      uint2 x[kSteps];
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        const int piece = 4 * (ks / (kPer / 4)) + t;
        x[ks] = real ? *reinterpret_cast<const uint2*>(q + piece * kPer + 4 * (ks % (kPer / 4))) : make_uint2(0u, 0u);
      }
      if constexpr (kScaled) {
        float sc = p.scale_log2;
        if (p.q_bf16) {
          // bf16 queries against f16 keys: to f16 after a power-of-two shift of the row, taken back in its scale
          float amax = 0.f;
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
            const uint32_t w[2] = {x[ks].x, x[ks].y};
#pragma unroll
            for (int u = 0; u < 2; ++u)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xFFFF0000u))));
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          int sh = 0;
          if (amax > 0.f && amax < INFINITY) {
            int e;
            frexpf(amax, &e);
            sh = max(-120, min(120, 12 - e));            // amax 2^sh in [2^11, 2^12): products and their sums stay in fp32
          }
          const float mul = __uint_as_float((uint32_t)(127 + sh) << 23);
          sc *= __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
            x[ks].x = pack2<false>(__uint_as_float(x[ks].x << 16) * mul, __uint_as_float(x[ks].x & 0xFFFF0000u) * mul);
            x[ks].y = pack2<false>(__uint_as_float(x[ks].y << 16) * mul, __uint_as_float(x[ks].y & 0xFFFF0000u) * mul);
          }
        }
        if (warp == 0 && t == 0) s_scale[8 * n + g] = sc;
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        qb[n][ks][0] = x[ks].x;
        qb[n][ks][1] = x[ks].y;
      }
    }
  }
  __syncthreads();                                       // s_lo, s_hi, s_scale
  if constexpr (kScaled) {
#pragma unroll
    for (int j = 0; j < kScales; ++j) scale[j] = s_scale[8 * (j >> 1) + 2 * t + (j & 1)];
  } else {
    scale[0] = p.scale_log2;
  }

  // rows 8 n + 2 t + e of this lane: j = 2 n + e
  float o[kMt][NT][4], m[2 * NT], l[2 * NT];
#pragma unroll
  for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
  }

  int stage = 0;
  for (int i = 0; i < n_groups; ++i) {
    cp_async_wait<T::kStages - 2>();
    __syncwarp();
    const bool skip = (bad >> stage) & 1u;
    const uint32_t sk = ring + (uint32_t)stage * T::kStage, sv = sk + T::kHalf;
    const int pos = begin + kGroup * (warp + kWarps * i);
    // the stage freed by the last iteration takes the group kStages - 1 ahead
    issue(i + T::kStages - 1, stage == 0 ? T::kStages - 1 : stage - 1);
    if (!skip) {
      // ------------------------------------------------------------ S^T = K Q^T: keys g, g + 8, rows 2t, 2t + 1
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      if constexpr (KV == kE2M1) {
        // a thread's bytes of a row: of each scale's group the two that hold its 4 dims, which make one k-step
        constexpr int kW = D / 32;                       // words: two groups each
        uint32_t w0[kW], w1[kW], c0[kW / 2], c1[kW / 2];
        const uint32_t ss = sk + 2 * T::kHalf;
        if constexpr (D == 128) {
          const uint4 k0 = lds128(sk + g * T::kRow + 16 * t), k1 = lds128(sk + (8 + g) * T::kRow + 16 * t);
          const uint2 s0 = lds64(ss + g * T::kScaleRow), s1 = lds64(ss + (8 + g) * T::kScaleRow);
          w0[0] = k0.x, w0[1] = k0.y, w0[kW - 2] = k0.z, w0[kW - 1] = k0.w;
          w1[0] = k1.x, w1[1] = k1.y, w1[kW - 2] = k1.z, w1[kW - 1] = k1.w;
          c0[0] = s0.x, c0[kW / 2 - 1] = s0.y;
          c1[0] = s1.x, c1[kW / 2 - 1] = s1.y;
        } else {
          const uint2 k0 = lds64(sk + g * T::kRow + 8 * t), k1 = lds64(sk + (8 + g) * T::kRow + 8 * t);
          w0[0] = k0.x, w0[1] = k0.y;
          w1[0] = k1.x, w1[1] = k1.y;
          c0[0] = lds32(ss + g * T::kScaleRow);
          c1[0] = lds32(ss + (8 + g) * T::kScaleRow);
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16x2x4(w0[j], x[0], x[1], x[2], x[3]);
          e2m1x8_to_f16x2x4(w1[j], y[0], y[1], y[2], y[3]);
          const uint32_t f0 = e4m3x2_to_f16x2((uint16_t)(c0[j / 2] >> (16 * (j & 1)))), f1 = e4m3x2_to_f16x2((uint16_t)(c1[j / 2] >> (16 * (j & 1))));
#pragma unroll
          for (int u = 0; u < 2; ++u) {                  // code x scale has 6 bits at most and is at least 2^-10: exact in f16
            const uint32_t a[4] = {mul_half(f0, u, x[2 * u]), mul_half(f1, u, y[2 * u]), mul_half(f0, u, x[2 * u + 1]), mul_half(f1, u, y[2 * u + 1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kB>(s[n], a, qb[n][2 * j + u][0], qb[n][2 * j + u][1]);
          }
        }
      } else
#pragma unroll
      for (int c4 = 0; c4 < T::kChunks / 4; ++c4) {
        const uint4 k0 = lds128(sk + T::k_at(g, 4 * c4 + t)), k1 = lds128(sk + T::k_at(8 + g, 4 * c4 + t));
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        if constexpr (KV == kE4M3) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)(w0[u] & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(w1[u] & 0xFFFFu)),
                                   e4m3x2_to_f16x2((uint16_t)(w0[u] >> 16)), e4m3x2_to_f16x2((uint16_t)(w1[u] >> 16))};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kB>(s[n], a, qb[n][4 * c4 + u][0], qb[n][4 * c4 + u][1]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a[4] = {w0[2 * u], w1[2 * u], w0[2 * u + 1], w1[2 * u + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kB>(s[n], a, qb[n][2 * c4 + u][0], qb[n][2 * c4 + u][1]);
          }
        }
      }
      // ------------------------------------------------------------ softmax, one pass
      if (pos < all_lo || pos + kGroup > all_hi) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int place = g + 8 * (e >> 1), r = 8 * n + 2 * t + (e & 1), key = pos + (KV == kE2M1 ? four_key(place) : place);
            if (key < s_lo[r] || key >= s_hi[r]) s[n][e] = -INFINITY;
          }
      }
      bool raise = false;
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j)                   // m = -inf: any logit raises it
        raise |= fmaf(fmaxf(s[j >> 1][j & 1], s[j >> 1][2 + (j & 1)]), scale[j % kScales], -m[j]) > kRaise + lift;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) {
          float mx = fmaxf(s[j >> 1][j & 1], s[j >> 1][2 + (j & 1)]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(fmaf(mx, scale[j % kScales], -lift), m[j]);
          const float f = (mx == -INFINITY) ? 1.f : ex2_ftz(m[j] - mx);   // m = -inf before: 0, on sums that are 0
          m[j] = mx;
          l[j] *= f;
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][j >> 1][j & 1] *= f;
            o[mt][j >> 1][2 + (j & 1)] *= f;
          }
        }
      }
      uint32_t pb[NT][2];                                // P^T: keys 2t, 2t + 1 and 2t + 8, 2t + 9 of row g
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * n + e;
          const float mu = m[j] == -INFINITY ? 0.f : m[j], sc = scale[j % kScales];
          w[e] = ex2_ftz(fmaf(s[n][e], sc, -mu));
          w[2 + e] = ex2_ftz(fmaf(s[n][2 + e], sc, -mu));
          l[j] += w[e] + w[2 + e];
        }
        pb[n][0] = movmatrix_trans(pack2<kB>(w[0], w[1]));
        pb[n][1] = movmatrix_trans(pack2<kB>(w[2], w[3]));
      }
      // ------------------------------------------------------------ O^T += V^T P^T
      if constexpr (KV == kE2M1) {
        // thread row g of tile mt is dim 16 mt + 2 g, row g + 8 the next one: byte g of each scale's group, of keys t, t + 4, t + 8, t + 12
        constexpr int kW = D / 64;                       // words of a thread's bytes of a key: 4 groups each
        uint32_t w[4][kW], c[4][kW];
        const uint32_t ss = sk + 2 * T::kHalf + T::kScales + 4 * t * T::kScaleRow;
        if constexpr (D == 128) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint2 x = lds64(sv + T::v_at(t + 4 * u, g >> 1) + 8 * (g & 1));
            w[u][0] = x.x, w[u][kW - 1] = x.y;
          }
          const uint4 x = lds128(ss), y = lds128(ss + 16);
          c[0][0] = x.x, c[0][kW - 1] = x.y, c[1][0] = x.z, c[1][kW - 1] = x.w;
          c[2][0] = y.x, c[2][kW - 1] = y.y, c[3][0] = y.z, c[3][kW - 1] = y.w;
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u][0] = lds32(sv + T::v_at(t + 4 * u, g >> 2) + 4 * (g & 3));
          const uint4 x = lds128(ss);
          c[0][0] = x.x, c[1][0] = x.y, c[2][0] = x.z, c[3][0] = x.w;
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          // codes and scales of two keys side by side, as the products take them
          uint32_t v[4][4], f[2][4];                     // [row g, row g + 8 of keys t, t + 4; of keys t + 8, t + 12][group]
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = w[2 * u][j], y = w[2 * u + 1][j];
            e2m1x8_to_f16x2x4((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), v[2 * u][0], v[2 * u][1], v[2 * u][2], v[2 * u][3]);
            e2m1x8_to_f16x2x4(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), v[2 * u + 1][0], v[2 * u + 1][1], v[2 * u + 1][2], v[2 * u + 1][3]);
            const uint32_t lo = __byte_perm(c[2 * u][j], c[2 * u + 1][j], 0x5140), hi = __byte_perm(c[2 * u][j], c[2 * u + 1][j], 0x7362);
            f[u][0] = e4m3x2_to_f16x2((uint16_t)(lo & 0xFFFFu));
            f[u][1] = e4m3x2_to_f16x2((uint16_t)(lo >> 16));
            f[u][2] = e4m3x2_to_f16x2((uint16_t)(hi & 0xFFFFu));
            f[u][3] = e4m3x2_to_f16x2((uint16_t)(hi >> 16));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a[4] = {mul_pair(v[0][e], f[0][e]), mul_pair(v[1][e], f[0][e]), mul_pair(v[2][e], f[1][e]), mul_pair(v[3][e], f[1][e])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kB>(o[4 * j + e][n], a, pb[n][0], pb[n][1]);
          }
        }
      } else if constexpr (KV == kE4M3) {
        // thread row g of tile mt is dim kPd g + 2 mt, row g + 8 the next one: rows 2t, 2t+1, 2t+8, 2t+9 of V
        constexpr int kPd = D / 8;
        uint32_t w[4][kPd / 4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = 2 * t + (u & 1) + 8 * (u >> 1);
          if constexpr (D == 128) {
            const uint4 x = lds128(sv + T::v_at(r, g));
            w[u][0] = x.x;
            w[u][1] = x.y;
            w[u][2] = x.z;
            w[u][3] = x.w;
          } else {
            const uint2 x = lds64(sv + T::v_at(r, g >> 1) + 8 * (g & 1));
            w[u][0] = x.x;
            w[u][1] = x.y;
          }
        }
#pragma unroll
        for (int n4 = 0; n4 < kPd / 4; ++n4) {
          const uint32_t a01 = __byte_perm(w[0][n4], w[1][n4], 0x5140), a23 = __byte_perm(w[0][n4], w[1][n4], 0x7362);
          const uint32_t c01 = __byte_perm(w[2][n4], w[3][n4], 0x5140), c23 = __byte_perm(w[2][n4], w[3][n4], 0x7362);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = u ? a23 : a01, y = u ? c23 : c01;
            const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)(x & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                                   e4m3x2_to_f16x2((uint16_t)(y & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(y >> 16))};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kB>(o[2 * n4 + u][n], a, pb[n][0], pb[n][1]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          uint32_t r4[4];
          ldmatrix_x4_trans(sv + T::v_at(lane & 15, 2 * mt + (lane >> 4)), r4);
          const uint32_t a[4] = {r4[0], r4[2], r4[1], r4[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<kB>(o[mt][n], a, pb[n][0], pb[n][1]);
        }
      }
    }
    __syncwarp();                        // every lane has read the stage before it is filled again
    stage = stage + 1 == T::kStages ? 0 : stage + 1;
  }

  // ---------------------------------------------------------------- merge the warps
  cp_async_wait<0>();
  __syncwarp();
  float* so = reinterpret_cast<float*>(sm + (size_t)warp * T::kRing);   // [row][kOutLd]
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    const int r = 8 * (j >> 1) + 2 * t + (j & 1);
    if (g == 0) {
      s_m[warp][r] = m[j];
      s_l[warp][r] = l[j];
    }
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        so[r * T::kOutLd + (KV == kE4M3 ? D / 8 * g + 2 * mt + u : KV == kE2M1 ? 16 * mt + 2 * g + u : 16 * mt + g + 8 * u)] = o[mt][j >> 1][2 * u + (j & 1)];
  }
  __syncthreads();
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
    float4* mine = reinterpret_cast<float4*>(sm + ((size_t)r * T::kOutLd + 4 * d4) * 4);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      add(a, L, M, s_m[w][r], s_l[w][r], *reinterpret_cast<const float4*>(reinterpret_cast<uint8_t*>(mine) + (size_t)w * T::kRing));
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
        const uint32_t x = cluster_map(o_at + ((uint32_t)r * T::kOutLd + 4 * d4) * 4, c);
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

// The splits of one row, joined in a fixed order: o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
// A lane per D / 32 dims; a few KB per row and split, so what counts is that the loads of several splits are
// in flight at once: unrolled by 4, and by W warps per row, each of which takes every W-th split.
constexpr int kJoinWide = 8;             // warps per row for more than this many splits, else one
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) paged_join_kernel(const __grid_constant__ PagedAttnParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = p.nq * p.group;
  const int64_t id = W == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;         // (b, h, row)
  const int first_split = W == 1 ? 0 : warp;
  if (id >= (int64_t)p.batch * p.heads * rows) return;
  const int row = (int)(id % rows);
  const int64_t bh = id / rows;
  const int b = (int)(bh / p.heads), h = (int)(bh % p.heads);
  const Span sp = request_span(p, b);
  if (sp.used == 1) return;              // written by its only split
  constexpr int V = D / 32;
  const int64_t first = bh * p.n_splits * rows + row;
  float M = -INFINITY;
  for (int c = lane; c < sp.used; c += 32) M = fmaxf(M, __ldcg(p.part_ml + 2 * (first + (int64_t)c * rows)));
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float a[V], L = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int c = first_split; c < sp.used; c += W) {
    const int64_t at = first + (int64_t)c * rows;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * at));
    float x[V];
    if constexpr (V == 4) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + lane);
      x[0] = y.x;
      x[1] = y.y;
      x[V - 2] = y.z;
      x[V - 1] = y.w;
    } else {
      const float2 y = __ldcg(reinterpret_cast<const float2*>(p.part_o + at * D) + lane);
      x[0] = y.x;
      x[1] = y.y;
    }
    if (ml.x != -INFINITY || ml.y != 0.f) {
      const float f = ml.x == -INFINITY ? 0.f : ex2_ftz(ml.x - M);
      L += f * ml.y;
#pragma unroll
      for (int e = 0; e < V; ++e) a[e] += f * x[e];
    }
  }
  if constexpr (W > 1) {                 // the warps' sums, in order
    __shared__ float s_sum[W][V + 1][32];
#pragma unroll
    for (int e = 0; e < V; ++e) s_sum[warp][e][lane] = a[e];
    s_sum[warp][V][lane] = L;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
#pragma unroll
      for (int e = 0; e < V; ++e) a[e] += s_sum[w][e][lane];
      L += s_sum[w][V][lane];
    }
  }
  const int64_t at = ((int64_t)b * p.nq + row / p.group) * p.heads_q + h * p.group + row % p.group;
  const float inv = L != 0.f ? p.v_scale / L : 0.f;
  uint32_t y[V / 2];
#pragma unroll
  for (int e = 0; e < V; e += 2)
    y[e / 2] = p.q_bf16 ? pack2<true>(a[e] * inv, a[e + 1] * inv) : pack2<false>(a[e] * inv, a[e + 1] * inv);
  uint16_t* out = p.out + at * D + V * lane;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[V / 2 - 1]);
  else
    *reinterpret_cast<uint32_t*>(out) = y[0];
  if (p.lse && lane == 0) p.lse[at] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int D, int KV, int NT, bool CLUSTER>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t s) {
  auto kernel = paged_attn_kernel<D, KV, NT, CLUSTER>;
  constexpr size_t smem = (size_t)kWarps * Tile<D, KV, NT>::kRing;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_splits * p.batch * p.heads * p.chunks);
  cfg.blockDim = dim3(kThreads);
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
template <int D, int KV>
cudaError_t launch_nt(const PagedAttnParams& p, cudaStream_t s) {
  switch ((p.chunk_rows + 7) / 8) {
    case 1: return p.cluster ? launch<D, KV, 1, true>(p, s) : launch<D, KV, 1, false>(p, s);
    case 2: return p.cluster ? launch<D, KV, 2, true>(p, s) : launch<D, KV, 2, false>(p, s);
    case 3: return p.cluster ? launch<D, KV, 3, true>(p, s) : launch<D, KV, 3, false>(p, s);
  }
  static_assert(kTcRows <= 3 * 8, "four tiles only for pages of 8 and 4 bits");
  if constexpr (KV == kE4M3 || KV == kE2M1)
    return p.cluster ? launch<D, KV, 4, true>(p, s) : launch<D, KV, 4, false>(p, s);
  else
    return cudaErrorInvalidValue;
}
template <int D>
cudaError_t launch_kv(const PagedAttnParams& p, int kv, cudaStream_t s) {
  switch (kv) {
    case kBf16: return launch_nt<D, kBf16>(p, s);
    case kF16: return launch_nt<D, kF16>(p, s);
    case kE4M3: return launch_nt<D, kE4M3>(p, s);
    default: return launch_nt<D, kE2M1>(p, s);
  }
}

}  // namespace

// Splits by rounds of the `places` that the GPU has for CTAs: the n with the least rounds x (keys of a job + 400) + 20 n,
// in the time of a key. A job costs what 400 keys do besides its own (its start and end), a split 20 in the join; a
// round that is not full costs as much as a full one. In w rounds the best n is the largest that fits.
struct Rounds {
  int64_t places;
  int64_t count;                         // numbers of rounds looked at
  bool few;                              // no more splits than where the two last terms meet
  int64_t first(int64_t ctas) const { return (ctas + places - 1) / places; }
  int64_t splits_in(int64_t w, int64_t ctas, int64_t span) const {
    int64_t n = imin64(places * w / ctas, (span + 127) / 128);
    if (few) n = imin64(n, (int64_t)sqrtf((float)(w * span) / 20.f));
    return imax64(1, n);
  }
  int64_t most(int64_t ctas, int64_t span) const { return splits_in(first(ctas) + count - 1, ctas, span); }
};
// The tcgen05 kernel, one CTA to an SM. 64 requests x 4 heads x 16,384 keys, ragged: n = 1, 4, 9: 246, 204, 229 us;
// x 4,097: 73, 77, 105; 8 x 4 x 16,384: n = 3, 4, 5, 9: 54.6, 53.9, 74.5, 59.0
constexpr Rounds kTcRounds = {kSms, 8, true};
// The warp MMA kernel with 17 to 32 rows, two to an SM. Against as many CTAs as four to an SM would be, in no rounds: 16
// requests x 8 heads x 20 rows, f16, 4,097 keys 30 us (46), 16,384 97 (115); 16 x 4 x 35 rows, E4M3, 4,097 36 (40), 16,384 93 (98);
// 64 x 4 x 24 rows, bf16, of 1 .. 16,384 keys 187 (206), all 65,536 1,240 (1,205); 4 x 4 x 35, E4M3, 4,097 17.1 (15.9)
constexpr Rounds kWideRounds = {2 * kSms, 6, false};
static int64_t best_splits(const Rounds& r, int64_t ctas, int64_t span) {
  int64_t best = 1, cost = INT64_MAX;
  for (int64_t w = r.first(ctas); w < r.first(ctas) + r.count; ++w) {
    const int64_t n = r.splits_in(w, ctas, span);
    const int64_t c = r.first(ctas * n) * (span / n + 400) + 20 * n;
    if (c < cost) {
      cost = c;
      best = n;
    }
  }
  return best;
}

// Which kernel, query rows per CTA and splits of the length.
// 16-bit pages and more than kTcRows query rows take the tcgen05 kernel, up to 128 rows (whole queries) to a CTA. There and
// in the warp MMA kernel, 64 requests x 4 heads of 128 dims, of 1 .. 8,192 keys: 32 rows 105 and 164 us, 24 rows 104 and 124;
// 1,000 keys: 33.3 and 33.1, 33.5 and 28.6; 1 request x 8 heads x 1,000 keys: 13.0 and 12.4, 13.0 and 9.9; 16 x 8 x 8,192 keys of 64
// dims: 28 rows 59.7 and 55.1, 18 rows 59.8 and 47.7. Else up to 32 rows one CTA reads its keys once for all of them; more rows
// (E4M3) are dealt out evenly (35: 18 and 17), and the later CTAs' keys come from L2.
// Up to 16 rows the splits make about as many CTAs as the GPU holds at a time, 3 per SM: more only add starts and joins (4
// requests of 131,072 FP8 keys: 168 us with 448 CTAs, 193 with 608, 217 with 1,216); from 17 rows on rounds of 2 per SM
// decide. No split is shorter than 256 keys (8 per group of a warp; in a cluster 128).
// Splits that all run at a time join in clusters (1 request of 1,000 keys: 6.7 us against 8.5); with more
// CTAs than that, a cluster's short CTAs would hold places until its longest ends (32 ragged contexts: 99
// us against 93).
// A request's splits follow from max_vis and the sizes alone, so that its result does not depend on
// where it stands in the batch. (Equal pieces of all requests' keys, one per place on the GPU, were
// slower: 109 against 94 us for 32 ragged contexts, because SMs do not get equal shares of HBM.)
static bool wide(const PagedSplit& s) { return !s.tc && s.chunk_rows > 16; }
PagedSplit paged_split(int32_t batch, int32_t heads, int32_t group, int32_t nq, int64_t max_vis, int32_t window, int32_t kv_dtype) {
  PagedSplit s;
  const int32_t rows = nq * group;
  s.tc = (kv_dtype == HSA_BF16 || kv_dtype == HSA_F16) && rows > kTcRows;
  if (s.tc) {
    const int32_t queries = nq < 128 / group ? nq : 128 / group;
    s.chunks = (nq + queries - 1) / queries;
    s.chunk_rows = queries * group;
  } else {
    s.chunks = (rows + 31) / 32;
    s.chunk_rows = (rows + s.chunks - 1) / s.chunks;
  }
  s.align = s.tc ? 64 : 16;
  int64_t span = max_vis;
  if (window > 0 && (int64_t)window + nq + s.align - 1 < span) span = (int64_t)window + nq + s.align - 1;   // vis one apart, as in a draft
  const int64_t ctas = (int64_t)batch * heads * s.chunks, places = kSms * ctas_per_sm((s.chunk_rows + 7) / 8);
  int64_t n;
  if (s.tc) {
    n = best_splits(kTcRounds, ctas, span);
  } else {
    const int64_t most = wide(s) ? best_splits(kWideRounds, ctas, span) : (places + ctas / 2) / ctas;
    n = imin64(most, (span + 255) / 256);
    if (n < 8) n = imin64(imin64(most, 8), (span + 127) / 128);
  }
  n = imax64(1, n);
  s.n_splits = (int32_t)n;
  s.split_len = (int32_t)imax64(64, ((span + n - 1) / n + 63) / 64 * 64);
  s.cluster = !s.tc && n > 1 && n <= 8 && ctas * n <= places;
  s.joined = n > 1 && !s.cluster;
  return s;
}

// The most splits that leave their parts in the workspace, for any length up to max_vis and any window
int64_t paged_splits_most(int32_t batch, int32_t heads, int32_t group, int32_t nq, int64_t max_vis, int32_t kv_dtype) {
  const PagedSplit s = paged_split(batch, heads, group, nq, max_vis, 0, kv_dtype);
  if (!s.tc && !wide(s)) return s.joined ? s.n_splits : 0;             // the longest has the most
  return (s.tc ? kTcRounds : kWideRounds).most((int64_t)batch * heads * s.chunks, max_vis);
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, const PagedSplit& sp, int32_t head_dim, int32_t kv_dtype, uint64_t wait_ns,
                              cudaStream_t s) {
  const cudaError_t e = sp.tc             ? launch_paged_rows(p, head_dim, kv_dtype, wait_ns, s)
                        : head_dim == 128 ? launch_kv<128>(p, kv_dtype, s)
                                          : launch_kv<64>(p, kv_dtype, s);
  if (e != cudaSuccess || !sp.joined) return e;
  const int64_t ids = (int64_t)p.batch * p.heads * p.nq * p.group;
  if (p.n_splits > kJoinWide) {
    const dim3 grid((unsigned)ids), block(32 * kJoinWide);
    return head_dim == 128 ? launch_pdl(paged_join_kernel<128, kJoinWide>, grid, block, 0, s, p)
                           : launch_pdl(paged_join_kernel<64, kJoinWide>, grid, block, 0, s, p);
  }
  const dim3 grid((unsigned)((ids + 3) / 4));
  return head_dim == 128 ? launch_pdl(paged_join_kernel<128, 1>, grid, dim3(128), 0, s, p)
                         : launch_pdl(paged_join_kernel<64, 1>, grid, dim3(128), 0, s, p);
}

}  // namespace hsa
