// Causal attention over packed prompts with grouped heads (hsa_prompt_attn):
//   o_i = sum_j softmax_j(scale q_i.k_j) v_j over the keys j a query sees.
//
// Bound: the two products, 4 d flops per visible (query, key) pair and head, on the tensor cores;
// the exponentials and the rest of the softmax run beside them. One CTA takes two tiles of 128
// rows. A row is one query head of one token: the `group` heads that share a key-value head stand
// together (tt = 128 / group tokens per tile), so that grouped heads share every key tile and a
// tile spans few tokens, which keeps the masked part at the diagonal small.
//  - one warp loads Q once and 128-key tiles of K and V into a ring by TMA (128-byte swizzle);
//  - one thread issues the tcgen05 products: S_t = Q_t K^T (128 x 128, fp32 in tensor memory), then
//    O_t += P_t V with P_t read from tensor memory and V as an MN-major operand. In order:
//    PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1), so each tile's softmax runs while the tensor core works
//    on the other tile;
//  - two warp groups do the softmax of one tile each, one row per thread (no shuffles): the
//    running maximum and sum in fp32, P rounded to the operand type over S's columns. The maximum
//    is only raised, and O rescaled in tensor memory, when a logit passes it by 2^8; after the
//    first tiles that hardly happens, so the rescaling needs no warps of its own;
//  - keys come from the diagonal downwards, so the first tile already holds each row's own key;
//  - one warp clears the rows of V past the end of the sequence in its last tile: their weights
//    are zero, but zero times another sequence's infinity would not be.
// TMEM: S_0, S_1 (128 columns each, P over the first 64), O_0, O_1 (head_dim columns each).
// Every wait is bounded; a role that gives up leaves its loop, and the others follow at their
// next wait.
#include "hsa_common.cuh"
#include "hsa_internal.h"
#include "hsa_tc.cuh"

namespace hsa {
namespace {

constexpr int kTile = 128;               // rows of a query tile, keys of a key tile
constexpr int kSoftWarps = 8;            // 4 per query tile: two warp groups; the third holds the other roles
constexpr int kMmaWarp = 8, kLoadWarp = 9, kClearWarp = 10;
constexpr int kThreads = 12 * 32;
// registers per thread: 168 at launch (65,536 over 384 threads, in steps of 8), then 208 for the
// softmax groups, whose threads hold a row of 128 logits, and 88 for the third: 2 x 208 + 88 = 3 x 168
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "setmaxnreg draws on the launch's registers");
constexpr uint32_t kBlock = kTile * 128; // 64 dims of 128 rows, 128 bytes a row
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;            // log2 of how far a logit may pass the running maximum

struct PromptParams {
  CUtensorMap qm, km, vm;
  int32_t batch, heads_q, heads_kv, group, tt, window;
  int64_t n_q, n_k, out_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  float scale_log2;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  uint64_t wait_ns;
};

template <int D>
struct Shape {
  static constexpr uint32_t kTileBytes = (D / 64) * kBlock;      // of Q, K or V
  static constexpr int kStages = D == 128 ? 4 : 6;               // K and V tiles in turn
  static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kTileBytes, kOffMisc = kOffKv + kStages * kTileBytes;
  static constexpr uint32_t kSmem = kOffMisc + 256 + 1024;       // + alignment slack
};

__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u));
}
#define TMEM_ST32(taddr, r)                                                                                     \
  asm volatile(                                                                                                 \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"  \
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),                          \
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),        \
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),           \
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),           \
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)                        \
      : "memory")
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What a CTA works on: sequence b, tokens [i0, i0 + n) of its lq, and the key tiles of each query tile
struct Job {
  int b, i0, n, off;                     // off = lk - lq: token i stands at position i + off
  int q0, k0, lk;
  int jlo[2], jhi[2];                    // key tiles [jlo, jhi) of query tile t; empty: jlo = jhi = 0
};

// Tiles of the sequences in order, the last tiles (the most keys) of each first. One warp; `found`
// false: no such tile. With `check_all`, sequences past the tile are looked at too, for their bounds.
__device__ __forceinline__ bool find_job(const PromptParams& p, int64_t tile, bool check_all, Job& job) {
  const int lane = threadIdx.x & 31, tpc = 2 * p.tt;
  int64_t before = 0;
  bool found = false;
  for (int base = 0; base < p.batch && (!found || check_all); base += 32) {
    const int b = base + lane;
    int q0 = 0, lq = 0, k0 = 0, lk = 0;
    if (b < p.batch) {
      const int q1 = p.cu_q[b + 1], k1 = p.cu_k[b + 1];
      q0 = p.cu_q[b];
      k0 = p.cu_k[b];
      if (q0 >= 0 && q0 <= q1 && q1 <= p.n_q && k0 >= 0 && k0 <= k1 && k1 <= p.n_k) {
        lq = q1 - q0;
        lk = k1 - k0;
      } else {
        flag_status(p.status, HSA_FLAG_INDEX_RANGE);
      }
    }
    const int tiles = (lq + tpc - 1) / tpc;
    int64_t upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    upto += before;
    const uint32_t past = __ballot_sync(0xffffffffu, upto > tile);
    if (past && !found) {
      const int src = __ffs(past) - 1;
      const int64_t end = __shfl_sync(0xffffffffu, upto, src);
      job.b = base + src;
      job.q0 = __shfl_sync(0xffffffffu, q0, src);
      job.k0 = __shfl_sync(0xffffffffu, k0, src);
      job.lk = __shfl_sync(0xffffffffu, lk, src);
      const int l = __shfl_sync(0xffffffffu, lq, src);
      job.i0 = (int)(end - 1 - tile) * tpc;
      job.n = min(tpc, l - job.i0);
      job.off = job.lk - l;
      found = true;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  if (!found) return false;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = min(p.tt, job.n - t * p.tt), first = job.i0 + t * p.tt + job.off;   // first position
    const int hi = first + n;                                                         // past the last position
    job.jlo[t] = job.jhi[t] = 0;
    if (n > 0 && hi > 0) {
      job.jhi[t] = (hi + kTile - 1) / kTile;
      job.jlo[t] = p.window > 0 ? max(first - p.window + 1, 0) / kTile : 0;
    }
  }
  return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
  using L = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t sQ = base + L::kOffQ, sKv = base + L::kOffKv;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kOffMisc);
  uint32_t* s_tmem = misc;
  // mbarriers: q_full[2], s_full[2], p_full[2], o_full[2], cleared, drain, then kv_full[stage], kv_empty[stage]
  const uint32_t bars = smem_u32(misc + 2);
  const uint32_t q_full = bars, s_full = bars + 16, p_full = bars + 32, o_full = bars + 48, cleared = bars + 64,
                 drain = bars + 72, kv_full = bars + 80, kv_empty = kv_full + 8 * L::kStages;
  static_assert(8 + 80 + 16 * L::kStages <= 256, "barriers");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(s_tmem), 512);
  if (tid == 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + 8 * t, 1);
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 8 * t, 4);
      mbar_init(o_full + 8 * t, 1);
    }
    mbar_init(cleared, 1);
    mbar_init(drain, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 1);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(s_tmem);
  griddep_wait();
  griddep_launch_dependents();

  const int h = blockIdx.x % p.heads_kv;
  Job job = {};
  // every warp looks its job up itself (the same loads): no broadcast, no block barrier
  const bool any = find_job(p, blockIdx.x / p.heads_kv, blockIdx.x == gridDim.x - 1, job);
  const int j_top = max(job.jhi[0], job.jhi[1]);
  const int j_bot = min(job.jhi[0] > job.jlo[0] ? job.jlo[0] : 0x7fffffff, job.jhi[1] > job.jlo[1] ? job.jlo[1] : 0x7fffffff);
  const bool clear = any && (int64_t)j_top * kTile > job.lk;      // the top tile reaches past the sequence
  auto active = [&](int t, int j) { return j >= job.jlo[t] && j < job.jhi[t]; };
  bool ok = true;

  if (!any) {
    // a CTA past the last tile
  } else if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loads
      if (lane == 0 && j_top > 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (job.jhi[t] > job.jlo[t]) {
            mbar_arrive_expect_tx(q_full + 8 * t, (D / 64) * (uint32_t)(p.tt * p.group) * 128u);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_4d(sQ + t * L::kTileBytes + c * kBlock, &p.qm, 64 * c, 0, h, job.q0 + job.i0 + t * p.tt, q_full + 8 * t);
          }
        int c = 0;                         // tiles loaded so far: K, V, K, V, ...
        for (int j = j_top - 1; j >= j_bot && ok; --j) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++c) {
            const int s = c % L::kStages;
            ok = ok && mbar_wait(kv_empty + 8 * s, ((c / L::kStages) & 1) ^ 1, p.wait_ns);
            if (!ok) break;
            mbar_arrive_expect_tx(kv_full + 8 * s, L::kTileBytes);
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
              tma_3d(sKv + s * L::kTileBytes + d * kBlock, kv ? &p.vm : &p.km, 64 * d, h, job.k0 + kTile * j, kv_full + 8 * s);
          }
        }
        // nothing of this CTA's may be in flight when it ends, whatever the other roles did
        for (int e = max(0, c - L::kStages); e < c; ++e)
          ok = mbar_wait(kv_full + 8 * (e % L::kStages), (e / L::kStages) & 1, p.wait_ns) && ok;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (job.jhi[t] > job.jlo[t]) ok = mbar_wait(q_full + 8 * t, 0, p.wait_ns) && ok;
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- products
      if (lane == 0 && j_top > 0) {
        const uint32_t id_qk = idesc_f16(128, 128, false, false, BF16), id_pv = idesc_f16(128, D, false, true, BF16);
        auto qk = [&](int t, int c) {
          const uint64_t a = sdesc(sQ + t * L::kTileBytes, 16u, 1024u), b = sdesc(sKv + (c % L::kStages) * L::kTileBytes, 16u, 1024u);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((k >> 2) * kBlock + (k & 3) * 32u) >> 4;
            umma_f16(tmem + 128 * t, a + o, b + o, id_qk, k > 0);
          }
          umma_commit(s_full + 8 * t);
        };
        auto pv = [&](int t, int c, bool acc) {
          const uint64_t b = sdesc(sKv + (c % L::kStages) * L::kTileBytes, kBlock, 1024u);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            umma_f16_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, b + ((k * 16u * 128u) >> 4), id_pv, acc || k > 0);
        };
        auto wait_kv = [&](int c) {
          ok = ok && mbar_wait(kv_full + 8 * (c % L::kStages), (c / L::kStages) & 1, p.wait_ns);
          tc_fence_after();
        };
        int n_p[2] = {0, 0};
        int c = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (job.jhi[t] > job.jlo[t]) ok = ok && mbar_wait(q_full + 8 * t, 0, p.wait_ns);
        wait_kv(0);
        if (ok) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (active(t, j_top - 1)) qk(t, 0);
          umma_commit(kv_empty);
        }
        for (int j = j_top - 1; j >= j_bot && ok; --j, c += 2) {
          wait_kv(c + 1);
          if (clear && j == j_top - 1) ok = ok && mbar_wait(cleared, 0, p.wait_ns);
          bool k_here = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (active(t, j) && ok) {
              ok = mbar_wait(p_full + 8 * t, n_p[t] & 1, p.wait_ns);
              tc_fence_after();
              if (ok) {
                pv(t, c + 1, n_p[t] > 0);
                if (j == job.jlo[t]) umma_commit(o_full + 8 * t);
              }
              ++n_p[t];
            }
            if (j - 1 >= j_bot && active(t, j - 1) && ok) {
              if (!k_here) wait_kv(c + 2);
              k_here = true;
              if (ok) qk(t, c + 2);
            }
          }
          umma_commit(kv_empty + 8 * ((c + 1) % L::kStages));
          if (j - 1 >= j_bot) umma_commit(kv_empty + 8 * ((c + 2) % L::kStages));
        }
        umma_commit(drain);
        ok = mbar_wait(drain, 0, p.wait_ns) && ok;
      }
    } else if (warp == kClearWarp) {
      // ---------------------------------------------------------------- V past the sequence's end
      if (clear && j_top > 0) {
        ok = mbar_wait(kv_full + 8, 0, p.wait_ns);           // the top tile's V is the ring's second tile
        const int first = job.lk - kTile * (j_top - 1);
        if (ok) {
          for (int e = first * 8 + lane; e < kTile * 8; e += 32)
#pragma unroll
            for (int d = 0; d < D / 64; ++d) sts128(sKv + L::kTileBytes + d * kBlock + e * 16u, 0u, 0u, 0u, 0u);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(cleared);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------- softmax: one row per thread
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128u * t, tO = tmem + lanes + 256u + 128u * t;
    const int tok = t * p.tt + r / p.group;
    const bool real = r < p.tt * p.group && tok < job.n;
    const int pos = job.i0 + tok + job.off;
    const int hi = real ? pos + 1 : 0, lo = real && p.window > 0 ? max(pos - p.window + 1, 0) : 0;
    // key tiles that every row of this query tile sees whole need no mask
    const int t_first = job.i0 + t * p.tt + job.off, t_last = job.i0 + min(job.n, (t + 1) * p.tt) - 1 + job.off;
    const int whole_hi = t_first + 1, whole_lo = p.window > 0 ? max(t_last - p.window + 1, 0) : 0;
    float m = -INFINITY, l = 0.f;
    const float scale = p.scale_log2, raise = kRaise / scale;
    const uint64_t scale2 = f2_pack(scale, scale);
    int n_s = 0;
    for (int j = job.jhi[t] - 1; j >= job.jlo[t] && ok; --j, ++n_s) {
      ok = mbar_wait(s_full + 8 * t, n_s & 1, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) TMEM_LD32(tS + 32 * c, s[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_regs_ready(s[c]);
      if (kTile * (j + 1) > whole_hi || kTile * j < whole_lo) {
        const int hr = hi - kTile * j, lr = lo - kTile * j;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= hr || c < lr) s[c >> 5][c & 31] = 0xFF800000u;   // -inf
      }
      float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        mx0 = fmaxf(mx0, __uint_as_float(s[0][c]));
        mx1 = fmaxf(mx1, __uint_as_float(s[1][c]));
        mx2 = fmaxf(mx2, __uint_as_float(s[2][c]));
        mx3 = fmaxf(mx3, __uint_as_float(s[3][c]));
      }
      const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
      if (__any_sync(0xffffffffu, mx > m + raise)) {
        const float mn = fmaxf(m, mx);
        const float f = mn == -INFINITY ? 1.f : ex2_ftz((m - mn) * scale);   // m = -inf before: 0, on sums that are 0
        m = mn;
        l *= f;
        if (n_s > 0) {                   // PV of the last tile is complete: S's barrier came after it
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            TMEM_LD32(tO + 32 * c, o);
            tmem_wait_ld();
            tmem_regs_ready(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            TMEM_ST32(tO + 32 * c, o);
          }
        }
      }
      const float mu = m == -INFINITY ? 0.f : m * scale;
      const uint64_t nmu2 = f2_pack(-mu, -mu);
      uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int e = 64 * half + 2 * c;
          float z0, z1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1])), scale2, nmu2),
                    z0, z1);
          const float p0 = ex2_ftz(z0), p1 = ex2_ftz(z1);
          if (c & 1)
            sum1 = f2_add(sum1, f2_pack(p0, p1));
          else
            sum0 = f2_add(sum0, f2_pack(p0, p1));
          pk[c] = pack2<BF16>(p0, p1);
        }
        TMEM_ST32(tS + 32 * half, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * t);
      float a, b;
      f2_unpack(f2_add(sum0, sum1), a, b);
      l += a + b;
    }
    // ---------------------------------------------------------------- O / l
    const bool keys = job.jhi[t] > job.jlo[t];
    if (keys) {
      ok = ok && mbar_wait(o_full + 8 * t, 0, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const int64_t row = (int64_t)job.q0 + job.i0 + tok;
    const int hq = h * p.group + r % p.group;
    uint16_t* out = p.out + row * p.out_stride + (int64_t)hq * D;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if (ok) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (keys) {
          TMEM_LD32(tO + 32 * c, o);
          tmem_wait_ld();
          tmem_regs_ready(o);
        }
        if (real) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float a = l != 0.f ? __uint_as_float(o[e + 2 * u]) * inv : 0.f;
              const float b = l != 0.f ? __uint_as_float(o[e + 2 * u + 1]) * inv : 0.f;
              y[u] = pack2<BF16>(a, b);
            }
            *reinterpret_cast<uint4*>(out + 32 * c + e) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (p.lse && real) p.lse[row * p.heads_q + hq] = l != 0.f ? (m * scale + log2f(l)) * kLn2 : -INFINITY;
    }
  }
  if (!ok) flag_status(p.status, HSA_FLAG_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's tensor-map encoder, looked up once through the runtime (no libcuda link)
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

template <int D, bool BF16>
cudaError_t launch(const PromptParams& p, unsigned blocks, cudaStream_t s) {
  auto kernel = prompt_attn_kernel<D, BF16>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), Shape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), Shape<D>::kSmem, s, p);
}

}  // namespace

cudaError_t launch_prompt_attn(const hsa_prompt_args& a, uint32_t* status, uint64_t wait_ns, cudaStream_t s) {
  const EncodeTiledFn encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  PromptParams p;
  memset(&p, 0, sizeof(p));
  p.batch = a.batch;
  p.heads_q = a.heads_q;
  p.heads_kv = a.heads_kv;
  p.group = a.heads_q / a.heads_kv;
  p.tt = kTile / p.group;
  p.window = a.window;
  p.n_q = a.n_q;
  p.n_k = a.n_k;
  p.out_stride = a.out_stride;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k ? a.cu_k : a.cu_q;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.status = status;
  p.wait_ns = wait_ns;
  const CUtensorMapDataType type = a.dtype == HSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t d = (cuuint64_t)a.head_dim;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  {
    // q as [token][key-value head][head of the group][dim]: a box is tt tokens x the group x 64 dims
    const cuuint64_t dims[4] = {d, (cuuint64_t)p.group, (cuuint64_t)p.heads_kv, (cuuint64_t)a.n_q};
    const cuuint64_t strides[3] = {2 * d, 2 * d * p.group, 2 * (cuuint64_t)a.q_stride};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.group, 1, (cuuint32_t)p.tt};
    if (encode(&p.qm, type, 4, const_cast<void*>(a.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    // k and v as [row][key-value head][dim]: a box is 128 rows x 64 dims. Without any rows the maps
    // are never used (no sequence has keys); they stand on q then.
    const cuuint64_t dims[3] = {d, (cuuint64_t)p.heads_kv, (cuuint64_t)(a.n_k > 0 ? a.n_k : 1)};
    const cuuint64_t strides[2] = {2 * d, 2 * (cuuint64_t)(i ? a.v_stride : a.k_stride)};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile};
    void* at = const_cast<void*>(a.n_k > 0 ? (i ? a.v : a.k) : a.q);
    if (encode(i ? &p.vm : &p.km, type, 3, at, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // at most n_q / (2 tt) whole tiles and one more per sequence, and no more than tokens
  const int64_t tiles = imin64(a.n_q / (2 * p.tt) + a.batch, a.n_q + 1);
  const int64_t blocks = tiles * p.heads_kv;
  if (blocks > (int64_t)0x7fffffff) return cudaErrorInvalidValue;
  if (a.head_dim == 128)
    return a.dtype == HSA_BF16 ? launch<128, true>(p, (unsigned)blocks, s) : launch<128, false>(p, (unsigned)blocks, s);
  return a.dtype == HSA_BF16 ? launch<64, true>(p, (unsigned)blocks, s) : launch<64, false>(p, (unsigned)blocks, s);
}

}  // namespace hsa
