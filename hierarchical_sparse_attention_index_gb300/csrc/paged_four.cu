// Attention of a few new tokens per request over 4-bit pages (hsa_paged_attn_decode, HSA_E2M1):
//   o = sum_j softmax_j(scale q.k_j) v_j,  k and v E2M1 codes times an E4M3 scale for each 16 dims,
// split over the cache's length and joined as in paged_attn.cu, whose layout of the work (a CTA per request, key-value head, up
// to 24 query rows and split; 4 warps with rings of their own; transposed warp MMAs; one-pass softmax) this kernel shares.
//
// Bound: a key and its value are 144 bytes at 128 dims, an eighth of what fp32 would be and 9/16 of E4M3, so the
// instructions that a warp spends on a key decide: at the copy rate 16 keys have 392 clocks of a scheduler. Codes become f16
// pairs by one conversion (2 clocks each on the unit that does integer work as well, 64 for 16 keys), times the group's
// scale (exact: 6 bits, at least 2^-10), which leaves little for anything else. Hence
//  - pages hold rows in the order of the fragments: of K a thread's codes are one 16-byte load whose bytes 2s, 2s + 1 are its
//    part of k-step s, which is one scale's group; of V one 8-byte load whose byte s is its row of group s;
//  - a product with V pairs two keys in a register, a byte holds two dims of one key: the nibbles of two keys are exchanged
//    before the conversion, 4 instructions for 8 pairs;
//  - scales are converted once per warp, not by each thread that needs them (4 and 8 times as often), those of V
//    in pairs of keys as the products take them, and come from shared memory;
//  - the keys of a piece are taken in the order t, t + 4 (four_key), so that every shared load is free of bank conflicts;
//  - two pieces of 16 keys go through a turn of the loop together: two independent chains, one vote and one wait for both.
// Fewer bits than 32 are in the weights, f16 for the product with V as in paged_attn.cu (a relative 2^-11 each, independent from key to
// key; the sums take them unrounded: an f16 result of 64 x 5 queries is off by 2.8e-4 of its size, 2.1e-4 with fp32 weights; bf16
// results by 1.7e-3 with either), and in bf16 queries, which become f16 by a power of two per row.
// Measured (8 rows, bf16 queries, 128 dims): 16 requests x 8 heads x 8,192 keys 37.1 us, 0.60 of the measured copy rate, 4 x 8 x
// 131,072 112 us, 0.80, 32 x 8 of 1 .. 8,192 keys 43.4 us, 1 x 8 x 1,000 6.6 us; 16 rows, 64 x 8 x 4,096 91.5 us; 64 dims, 8 rows, 32 x 8 x 8,192
// 42.7 us. In the long one the schedulers issue in 62 % of the clocks, 295 instructions for 16 keys; the integer and conversion unit is
// at 52 %, the tensor unit at 27 %, HBM at 79 %: what is left is waits between dependent instructions that 12 warps do not fill. With 16 rows
// there are 8 warps to an SM, which issue in 48 % (the tensor unit is at 35, HBM at 41). Of 1 .. 8,192 keys the CTAs start in the order of the
// grid, so that a long request's last splits start last: 768 CTAs for 456 places, issue 37 % over the whole launch.
#include "hsa_four.cuh"
#include "hsa_paged_warp.cuh"

namespace hsa {
namespace {

constexpr int kWarps = kPagedWarps, kThreads = kWarps * 32, kGroup = kPagedGroup;

// The key of a piece at place i of the products' key index, and back. Thread t's keys, places 2t, 2t + 1, 2t + 8 and 2t + 9, are
// then t, t + 4, t + 8, t + 12
__host__ __device__ __forceinline__ constexpr int four_key(int i) { return (i & 8) + ((i & 1) << 2) + ((i & 6) >> 1); }
__host__ __device__ __forceinline__ constexpr int four_place(int r) { return (r & 8) + ((r & 3) << 1) + ((r & 4) >> 2); }

__device__ __forceinline__ uint32_t mul_pair(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void sts128v(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Bytes of a warp's ring slot (one piece): K's codes, a row at its place in the products; V's codes, whose 16-byte chunks of rows
// t and t + 4 lie apart; K's and V's scales in the same orders. Behind the slots, the scales in f16 of the pieces of a turn.
template <int D, int NT>
struct Slot {
  static constexpr int kPieces = 2;                      // of a turn. One of 17 to 24 rows: 24 rows, 32 x 8 x 8,192 keys of 64 dims 80 us against 70
  static constexpr int kRow = D / 2, kChunks = kRow / 16, kHalf = kGroup * kRow;
  static constexpr int kScaleRow = D / 16, kScales = kGroup * kScaleRow;
  static constexpr int kBytes = 2 * kHalf + 2 * kScales;
  static constexpr int kCtas = four_ctas(NT, D);
  static constexpr int kSlots = D == 128 ? (NT <= 2 ? 6 : 10) : (NT == 1 ? 10 : NT == 2 ? 12 : 15);
  static constexpr int kWide = kPieces * 4 * kScales;    // f16 scales: of K, then of V
  static constexpr int kWarpBytes = kSlots * kBytes + kWide;
  static_assert(kCtas * (kWarps * kWarpBytes + 3 * 1024) <= 228 * 1024, "shared memory of an SM");
  static_assert(8 * NT * kPagedOutLd<D> * 4 <= kSlots * kBytes, "a warp's outputs fit its ring");
  static __host__ __device__ __forceinline__ constexpr uint32_t k_at(int r, int c) { return (uint32_t)(four_place(r) * kRow + c * 16); }
  static __host__ __device__ __forceinline__ constexpr uint32_t v_at(int r, int c) { return (uint32_t)(r * kRow + (kChunks == 4 ? c ^ (r & 2) : c) * 16); }
};

// NT: tiles of 8 query rows
// CLUSTER: the splits of a (request, head, chunk) are one cluster
template <int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, (Slot<D, NT>::kCtas)) paged_four_kernel(const __grid_constant__ PagedAttnParams p) {
  using T = Slot<D, NT>;
  constexpr int kSteps = D / 16, kMt = D / 16, kRows = 8 * NT, kP = T::kPieces;
  constexpr float lift = kLift<false>;                   // weights are 2^(x - m), m that much below the running maximum
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
  // Everything that depends on nothing but the block is asked for at once, before the first answer is needed: one wait on memory
  // before the first copies, not four: the rows' queries and lengths, the request's
  // lengths, and the pages of the warp's first pieces as they are unless a window or a length past max_vis moves them
  const int row0 = chunk * p.chunk_rows, row_end = min(row0 + p.chunk_rows, p.nq * p.group);
  uint2 qx[NT][kSteps];                  // k-step ks covers, of thread t, dims 16 ks + 4 t .. + 3
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 8 * n + g;
    const bool real = r < row_end;
    const int qi = real ? r / p.group : 0, hq = h * p.group + (real ? r % p.group : 0);
    const uint16_t* q = p.q + (((int64_t)b * p.nq + qi) * p.heads_q + hq) * D;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) qx[n][ks] = real ? *reinterpret_cast<const uint2*>(q + 16 * ks + 4 * t) : make_uint2(0u, 0u);
  }
  const bool real_row = lane < kRows && row0 + lane < row_end;
  const int raw_vis = real_row ? p.vis[(int64_t)b * p.nq + (row0 + lane) / p.group] : 0;
  const int likely = split * p.split_len, likely_pg = (likely + kGroup * (warp + kWarps * lane)) / p.page_size;
  const int likely_page = likely_pg < p.max_pages ? p.table[(int64_t)b * p.max_pages + likely_pg] : -1;
  const Span sp = request_span(p, b);
  if (!CLUSTER && split >= sp.used) return;
  const int begin = sp.base + split * sp.len, end = max(begin, min(begin + sp.len, sp.hi));   // keys of this CTA

  // ---------------------------------------------------------------- the ring: 16-key pieces of this warp, 64 keys apart
  const uint32_t ring = smem_u32(sm) + (uint32_t)warp * T::kWarpBytes, wide = ring + T::kSlots * T::kBytes;
  const int n_pieces = max(0, (end - begin + kGroup * (kWarps - warp) - 1) / (kGroup * kWarps));
  const int turns = (n_pieces + kP - 1) / kP;
  uint32_t bad = 0;                                      // bit i % 32: piece i is zeros
  const int64_t page_pieces = (int64_t)p.heads * (p.page_size / kGroup);
  // where 32 pieces lie, one per lane. Their pages are read a turn ahead of their use, and only read: looked at where they are
  // read, they would hold up the warp for as long as the table takes to answer
  auto page_of = [&](int of) {
    const int i = 32 * of + lane;
    return i < n_pieces ? p.table[(int64_t)b * p.max_pages + (begin + kGroup * (warp + kWarps * i)) / p.page_size] : -1;
  };
  auto pieces_of = [&](int of, int page) -> int64_t {
    const int i = 32 * of + lane, pos = begin + kGroup * (warp + kWarps * i);
    return i < n_pieces ? piece_at(p, sp, b, h, page_pieces, pos, pos / p.page_size, page) : 0;
  };
  int64_t pieces = pieces_of(0, begin == likely ? likely_page : page_of(0));
  int next_page = page_of(1);
  // this lane's copies of a piece: 16 bytes of every 32 / kChunks-th row of K and of V, and one row's scales, of K or of V
  constexpr int kCopies = kGroup * T::kChunks / 32;
  const int r0 = lane / T::kChunks, c0 = lane % T::kChunks, rs = lane & 15;
  const uint8_t* const k_src = p.k_pool + lane * 16;
  const uint8_t* const v_src = p.v_pool + lane * 16;
  const uint8_t* const s_src = (lane < 16 ? p.k_s : p.v_s) + rs * T::kScaleRow;
  const uint32_t k_dst = T::k_at(r0, c0), v_dst = T::kHalf + T::v_at(r0, c0);
  const uint32_t s_dst = 2 * T::kHalf + (uint32_t)(lane < 16 ? four_place(rs) : kGroup + rs) * T::kScaleRow;
  static_assert(T::kSlots - kP < 32, "the first copies are of the first 32 pieces");
  static_assert(kCopies == 1 || (T::k_at(8, 0) == 512 && T::v_at(8, 0) == 512), "rows 8 apart lie 512 bytes apart");
  const int issued = turns * kP;                         // the last turn's second piece may be none: zeros
  auto issue = [&](int i, uint32_t at) {                 // called with i = 0, 1, 2, ...; at: its slot
    const int64_t found = __shfl_sync(0xffffffffu, pieces, i & 31);
    if ((i & 31) == 31) {
      pieces = pieces_of((i >> 5) + 1, next_page);
      next_page = page_of((i >> 5) + 2);
    }
    if (i < issued) {
      const uint32_t seen = (uint32_t)found & 0xFFFFu;
      const uint64_t piece = (uint32_t)(found >> 16);    // fewer than 2^32: a piece has 576 bytes at least
      const uint8_t* k = k_src + piece * T::kHalf;
      const uint8_t* v = v_src + piece * T::kHalf;
      const uint8_t* sc = s_src + piece * T::kScales;
      if (seen == 0xFFFFu) {
        if (bad) bad &= ~(1u << (i & 31));
        page_copy_scales<T::kScaleRow>(at + s_dst, sc, T::kScaleRow);
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          page_copy16(at + k_dst + u * 512, k + u * 512);
          page_copy16(at + v_dst + u * 512, v + u * 512);
        }
      } else {
        // rows no query sees are not read: they become zeros, whatever the pool holds there
        bad = (bad & ~(1u << (i & 31))) | ((seen ? 0u : 1u) << (i & 31));
        const bool n = (seen >> rs) & 1u;
        page_copy_scales<T::kScaleRow>(at + s_dst, n ? sc : p.k_s, n ? (uint32_t)T::kScaleRow : 0u);
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          const uint32_t m = (seen >> (r0 + 8 * u)) & 1u ? 16u : 0u;
          page_copy16z(at + k_dst + u * 512, m ? k + u * 512 : p.k_pool, m);
          page_copy16z(at + v_dst + u * 512, m ? v + u * 512 : p.v_pool, m);
        }
      }
    }
    page_copies_commit();
  };
#pragma unroll
  for (int s = 0; s < T::kSlots - kP; ++s) issue(s, ring + s * T::kBytes);

  // ---------------------------------------------------------------- each row's keys, for masked pieces
  int all_lo = 0, all_hi = 0x7fffffff;                   // inside [all_lo, all_hi) no row masks anything
  if (lane < kRows) {
    int2 keys = make_int2(0, 0);
    if (real_row) {
      keys = keys_of(p, raw_vis, split == 0 && h == 0);
      all_lo = keys.x;
      all_hi = keys.y;
    }
    if (warp == 0) {
      s_lo[lane] = keys.x;
      s_hi[lane] = keys.y;
    }
  }
  all_lo = __reduce_max_sync(0xffffffffu, all_lo);
  all_hi = __reduce_min_sync(0xffffffffu, all_hi);

  // ---------------------------------------------------------------- queries into B fragments
  uint32_t qb[NT][kSteps][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float sc = p.scale_log2;
    if (p.q_bf16) queries_to_f16(qx[n], sc);
    if (warp == 0 && t == 0) s_scale[8 * n + g] = sc;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      qb[n][ks][0] = qx[n][ks].x;
      qb[n][ks][1] = qx[n][ks].y;
    }
  }
  __syncthreads();                                       // s_lo, s_hi, s_scale
  float scale[2 * NT];                                   // of rows 2t, 2t + 1 of each tile
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) scale[j] = s_scale[8 * (j >> 1) + 2 * t + (j & 1)];

  // rows 8 n + 2 t + e of this lane: j = 2 n + e
  float o[kMt][NT][4], m[2 * NT], mu[2 * NT], l[2 * NT]; // mu: m, or 0 where that is -inf
#pragma unroll
  for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    m[j] = -INFINITY;
    mu[j] = l[j] = 0.f;
  }

  // The scales that this lane converts: eight bytes, in two words of a slot, to 16 bytes of `wide`. 128 dims: lanes 0..15 a row of K
  // each, the others half the groups of a pair of V's keys t + 8u, t + 8u + 4. 64 dims: lanes 0..7 two rows of K, 8..15
  // a pair of V's keys, and 16 lanes more the second piece's.
  constexpr int kLanes = D / 4;                          // of a piece
  const int cv = lane % kLanes, vp = (cv - kLanes / 2) / (D / 64), cv_piece = lane / kLanes;
  const bool of_v = cv >= kLanes / 2;
  const uint32_t cv0 = 2 * T::kHalf + (of_v ? T::kScales + ((vp >> 1) + 8 * (vp & 1)) * T::kScaleRow + (D == 128 ? 4 * (cv & 1) : 0) : 8 * cv);
  const uint32_t cv1 = cv0 + (of_v ? 4 * T::kScaleRow : 4);
  const uint32_t sel0 = of_v ? 0x5140u : 0x3210u, sel1 = of_v ? 0x7362u : 0x7654u;
  auto widen_scales = [&](uint32_t slot_at, uint32_t to) {
    const uint32_t x = lds32(slot_at + cv0), y = lds32(slot_at + cv1);
    const uint32_t lo = __byte_perm(x, y, sel0), hi = __byte_perm(x, y, sel1);
    sts128v(to + cv * 16, make_uint4(e4m3x2_to_f16x2((uint16_t)(lo & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                                     e4m3x2_to_f16x2((uint16_t)(hi & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(hi >> 16))));
  };

  // turns [t0, t1) have no piece that a row does not see all of
  const int first = begin + kGroup * warp, span = kGroup * kWarps * kP;
  const int t0 = all_lo > first ? (all_lo - first + span - 1) / span : 0;
  const int t1 = all_hi < first + span - kGroup * (kWarps - 1) ? 0 : (all_hi - (first + span - kGroup * (kWarps - 1))) / span + 1;
  // slots of this turn's pieces, and those of the last one, which are free
  uint32_t slots[kP], freed[kP];
#pragma unroll
  for (int h2 = 0; h2 < kP; ++h2) {
    slots[h2] = ring + h2 * T::kBytes;
    freed[h2] = ring + (T::kSlots - kP + h2) * T::kBytes;
  }
  for (int i = 0; i < turns; ++i) {
    page_copies_wait<T::kSlots - 2 * kP>();
    __syncwarp();
    uint32_t none = 0;                   // bit h2: that piece of the turn is zeros
    if (bad) none = (bad >> (kP * i & 31)) & ((1u << kP) - 1u);
#pragma unroll
    for (int h2 = 0; h2 < kP; ++h2) issue(kP * i + T::kSlots - kP + h2, freed[h2]);
    if (none != (1u << kP) - 1u) {
      if constexpr (D == 128) {
#pragma unroll
        for (int h2 = 0; h2 < kP; ++h2) widen_scales(slots[h2], wide + h2 * 4 * T::kScales);
      } else {
        const int h2 = cv_piece % kP;                    // one piece: both halves of the warp do the same
        widen_scales(h2 ? slots[kP - 1] : slots[0], wide + h2 * 4 * T::kScales);
      }
      __syncwarp();
      // ------------------------------------------------------------ S^T = K Q^T: places g, g + 8, rows 2t, 2t + 1
      float s[kP][NT][4];
      constexpr int kKw = D / 32;                        // words of a thread's codes of a row: two groups each
      uint32_t w0[kP][kKw], w1[kP][kKw], f0[kP][kKw], f1[kP][kKw];
#pragma unroll
      for (int h2 = 0; h2 < kP; ++h2) {
        const uint32_t sk = slots[h2], sf = wide + h2 * 4 * T::kScales;
        if constexpr (D == 128) {
          const uint4 k0 = lds128(sk + g * T::kRow + 16 * t), k1 = lds128(sk + (8 + g) * T::kRow + 16 * t);
          const uint4 x0 = lds128(sf + g * 16), x1 = lds128(sf + (8 + g) * 16);
          w0[h2][0] = k0.x, w0[h2][1] = k0.y, w0[h2][kKw - 2] = k0.z, w0[h2][kKw - 1] = k0.w;
          w1[h2][0] = k1.x, w1[h2][1] = k1.y, w1[h2][kKw - 2] = k1.z, w1[h2][kKw - 1] = k1.w;
          f0[h2][0] = x0.x, f0[h2][1] = x0.y, f0[h2][kKw - 2] = x0.z, f0[h2][kKw - 1] = x0.w;
          f1[h2][0] = x1.x, f1[h2][1] = x1.y, f1[h2][kKw - 2] = x1.z, f1[h2][kKw - 1] = x1.w;
        } else {
          const uint2 k0 = lds64(sk + g * T::kRow + 8 * t), k1 = lds64(sk + (8 + g) * T::kRow + 8 * t);
          const uint2 x0 = lds64(sf + g * 8), x1 = lds64(sf + (8 + g) * 8);
          w0[h2][0] = k0.x, w0[h2][1] = k0.y;
          w1[h2][0] = k1.x, w1[h2][1] = k1.y;
          f0[h2][0] = x0.x, f0[h2][1] = x0.y;
          f1[h2][0] = x1.x, f1[h2][1] = x1.y;
        }
      }
#pragma unroll
      for (int j = 0; j < kKw; ++j)
#pragma unroll
        for (int h2 = 0; h2 < kP; ++h2) {                // two chains of products side by side
          uint32_t x[4], y[4];
          e2m1x8_to_f16x2x4(w0[h2][j], x[0], x[1], x[2], x[3]);
          e2m1x8_to_f16x2x4(w1[h2][j], y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a[4] = {mul_half(f0[h2][j], u, x[2 * u]), mul_half(f1[h2][j], u, y[2 * u]), mul_half(f0[h2][j], u, x[2 * u + 1]),
                                   mul_half(f1[h2][j], u, y[2 * u + 1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (j == 0 && u == 0)
                mma_f16_16816_zc(s[h2][n], a[0], a[1], a[2], a[3], qb[n][0][0], qb[n][0][1]);
              else
                mma16816<false>(s[h2][n], a, qb[n][2 * j + u][0], qb[n][2 * j + u][1]);
            }
          }
        }
      // ------------------------------------------------------------ softmax, one pass
      if (i < t0 || i >= t1 || none) {
#pragma unroll
        for (int h2 = 0; h2 < kP; ++h2) {
          const int pos = first + kGroup * kWarps * (kP * i + h2);
          const bool zeros = (none >> h2) & 1u;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 8 * n + 2 * t + (e & 1), key = pos + four_key(g + 8 * (e >> 1));
              if (key < s_lo[r] || key >= s_hi[r] || zeros) s[h2][n][e] = -INFINITY;
            }
        }
      }
      float top[2 * NT];
      bool raise = false;
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {                 // m = -inf: any logit raises it
        top[j] = fmaxf(s[0][j >> 1][j & 1], s[0][j >> 1][2 + (j & 1)]);
#pragma unroll
        for (int h2 = 1; h2 < kP; ++h2) top[j] = fmaxf(top[j], fmaxf(s[h2][j >> 1][j & 1], s[h2][j >> 1][2 + (j & 1)]));
        raise |= fmaf(top[j], scale[j], -m[j]) > kRaise + lift;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) {
          float mx = top[j];
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(fmaf(mx, scale[j], -lift), m[j]);
          const float f = (mx == -INFINITY) ? 1.f : ex2_ftz(m[j] - mx);   // m = -inf before: 0, on sums that are 0
          m[j] = mx;
          mu[j] = mx == -INFINITY ? 0.f : mx;
          l[j] *= f;
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][j >> 1][j & 1] *= f;
            o[mt][j >> 1][2 + (j & 1)] *= f;
          }
        }
      }
      uint32_t pb[kP][NT][2];                            // P^T: places 2t, 2t + 1 and 2t + 8, 2t + 9 of row g
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h2 = 0; h2 < kP; ++h2) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 2 * n + e;
            w[e] = ex2_ftz(fmaf(s[h2][n][e], scale[j], -mu[j]));
            w[2 + e] = ex2_ftz(fmaf(s[h2][n][2 + e], scale[j], -mu[j]));
            l[j] += w[e] + w[2 + e];
          }
          pb[h2][n][0] = movmatrix_trans(pack2<false>(w[0], w[1]));
          pb[h2][n][1] = movmatrix_trans(pack2<false>(w[2], w[3]));
        }
      // ------------------------------------------------------------ O^T += V^T P^T
      // thread row g of tile mt is dim 16 mt + 2 g, row g + 8 the next one: byte g of each scale's group, of keys t, t + 4, t + 8, t + 12
#pragma unroll
      for (int h2 = 0; h2 < kP; ++h2) {
        constexpr int kW = D / 64;                       // words of a thread's codes of a key: 4 groups each
        const uint32_t sv = slots[h2] + T::kHalf, sf = wide + h2 * 4 * T::kScales + 2 * T::kScales + t * 4 * T::kScaleRow * 2;
        uint32_t w[4][kW];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if constexpr (D == 128) {
            const uint2 x = lds64(sv + T::v_at(t + 4 * u, g >> 1) + 8 * (g & 1));
            w[u][0] = x.x, w[u][kW - 1] = x.y;
          } else {
            w[u][0] = lds32(sv + T::v_at(t + 4 * u, g >> 2) + 4 * (g & 3));
          }
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          // codes of two keys side by side, as the products take them, and their scales
          uint32_t v[4][4], f[2][4];                     // [row g, row g + 8 of keys t, t + 4; of keys t + 8, t + 12][group]
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = w[2 * u][j], y = w[2 * u + 1][j];
            e2m1x8_to_f16x2x4((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), v[2 * u][0], v[2 * u][1], v[2 * u][2], v[2 * u][3]);
            e2m1x8_to_f16x2x4(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), v[2 * u + 1][0], v[2 * u + 1][1], v[2 * u + 1][2], v[2 * u + 1][3]);
            const uint4 c = lds128(sf + (u * kW + j) * 16);
            f[u][0] = c.x, f[u][1] = c.y, f[u][2] = c.z, f[u][3] = c.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a[4] = {mul_pair(v[0][e], f[0][e]), mul_pair(v[1][e], f[0][e]), mul_pair(v[2][e], f[1][e]), mul_pair(v[3][e], f[1][e])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<false>(o[4 * j + e][n], a, pb[h2][n][0], pb[h2][n][1]);
          }
        }
      }
    }
    __syncwarp();                        // every lane has read the slots before they are filled again
#pragma unroll
    for (int h2 = 0; h2 < kP; ++h2) {
      freed[h2] = slots[h2];
      slots[h2] += kP * T::kBytes;
      if (slots[h2] >= ring + T::kSlots * T::kBytes) slots[h2] -= T::kSlots * T::kBytes;
    }
  }

  // ---------------------------------------------------------------- merge the warps
  page_copies_wait<0>();
  __syncwarp();
  float* so = reinterpret_cast<float*>(sm + (size_t)warp * T::kWarpBytes);   // [row][kPagedOutLd]
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
      for (int u = 0; u < 2; ++u) so[r * kPagedOutLd<D> + 16 * mt + 2 * g + u] = o[mt][j >> 1][2 * u + (j & 1)];
  }
  __syncthreads();
  merge_warps<D, NT, CLUSTER>(p, sp, b, h, split, row0, row_end, sm, T::kWarpBytes, s_m, s_l, s_part);
}

template <int D, int NT, bool CLUSTER>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t s) {
  return launch_splits<CLUSTER>(paged_four_kernel<D, NT, CLUSTER>, p, (size_t)kWarps * Slot<D, NT>::kWarpBytes, s);
}
template <int D>
cudaError_t launch_nt(const PagedAttnParams& p, cudaStream_t s) {
  switch ((p.chunk_rows + 7) / 8) {
    case 1: return p.cluster ? launch<D, 1, true>(p, s) : launch<D, 1, false>(p, s);
    case 2: return p.cluster ? launch<D, 2, true>(p, s) : launch<D, 2, false>(p, s);
    case 3: return p.cluster ? launch<D, 3, true>(p, s) : launch<D, 3, false>(p, s);
  }
  static_assert(kPagedTcRows <= 3 * 8, "no more tiles");
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_four(const PagedAttnParams& p, int32_t head_dim, cudaStream_t s) {
  return head_dim == 128 ? launch_nt<128>(p, s) : launch_nt<64>(p, s);
}

}  // namespace hsa
