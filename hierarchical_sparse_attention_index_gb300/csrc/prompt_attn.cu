// Causal attention over packed prompts with grouped heads (hsa_prompt_attn):
//   o_i = sum_j softmax_j(scale q_i.k_j) v_j over the keys j a query sees.
//
// Bound: the two products, 4 d flops per visible (query, key) pair and head, on the tensor cores;
// the exponentials and the rest of the softmax run beside them. One CTA per SM takes two tiles of
// 128 rows at a time. A row is one query head of one token: the `group` heads that share a key-value
// head stand together (tt = 128 / group tokens per tile), so that grouped heads share every key tile
// and a tile spans few tokens, which keeps the masked part at the diagonal small.
//  - CTAs stay and take the next block's work themselves (cluster launch control), while the loads
//    of the next work already run; the first work has the most keys;
//  - one warp loads Q, and 64-key tiles of K and V into a ring, by TMA (128-byte swizzle);
//  - a warp per query tile issues its tcgen05 products: S = Q K^T (128 x 64, fp32 in tensor memory,
//    two buffers, one key tile ahead), then O += P V with P read from tensor memory and V as an
//    MN-major operand. So S of the next key tile is there when the softmax comes to it. (A product
//    for 64 keys reads 6 KB of shared memory in the 32 clocks that it computes, 128 bytes a clock
//    can be read; one for 128 keys reads 8 KB in 64, but leaves room for one buffer only: 16,384
//    tokens took the same time, packed prompts 15 % more);
//  - a warp group does the softmax of each tile, one row per thread (no shuffles): the running
//    maximum and sum in fp32, P rounded to the operand type (a relative 2^-9 in bf16, 2^-12 in f16,
//    independent from key to key) over S's columns. The maximum is only raised, and O rescaled in
//    tensor memory, when a logit passes it by 2^8: weights stay below 256, and after the first
//    tiles that hardly happens, so the rescaling needs no warps of its own;
//  - keys come from the diagonal downwards, so the first tile already holds each row's own key;
//  - the rows of V's tiles that are no keys of the sequence are cleared before use: their weights
//    are zero, but zero times another sequence's infinity would not be.
// TMEM: S 2 x 64 columns per query tile (P over the first half of its buffer), O head_dim columns each.
// Every wait is bounded; a role that gives up leaves its loop, and the others follow at their next
// wait.
// Measured (16,384 tokens, 32 heads over 4, 128 dims): 1,444 us, 1,523 TFLOP/s, 0.79 of the measured
// bf16 peak; without the softmax's part 1,340 us, where shared memory bounds the products.
#include "hsa_flash.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kTile = 128;               // rows of a query tile
constexpr int kKeys = 64;                // keys of a key tile
constexpr int kSoftWarps = 8;            // 4 per query tile: two warp groups; the third holds the other roles
constexpr int kMmaWarp = 8, kLoadWarp = 10;              // a warp per query tile's products; warp 11 finds the work
constexpr int kThreads = 12 * 32;
// registers per thread: 168 at launch (65,536 over 384 threads, in steps of 8), then 208 for the
// softmax groups, whose threads hold a row of 128 logits, and 88 for the third: 2 x 208 + 88 = 3 x 168
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "setmaxnreg draws on the launch's registers");
constexpr uint32_t kBlockQ = kTile * 128, kBlockK = kKeys * 128;   // 64 dims of a tile, 128 bytes a row

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
  static constexpr uint32_t kQBytes = (D / 64) * kBlockQ, kKvBytes = (D / 64) * kBlockK;
  static constexpr int kStages = 8;                              // tiles of K and V in the ring
  static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kQBytes, kOffStage = kOffKv + kStages * kKvBytes;
  static constexpr uint32_t kSmem = kOffStage + kSoftWarps * 2048 + 1024;   // + alignment slack
};

// One piece of work: tokens [i0, i0 + n) of a sequence for key-value head h, as two query tiles, and
// the key tiles of each. Key tile j holds the keys kbase + 64 j ..; kbase is 0, or, with a window,
// such that the top tile ends at the last key (so that a window of w meets as few tiles as it can).
struct Job {
  int h, i0, n, off;                     // off = lk - lq: token i stands at position i + off
  int q0, k0, lk, kbase;
  int jlo[2], jhi[2];                    // key tiles [jlo, jhi) of query tile t; empty: jlo = jhi = 0
  int clear_j, clear_lo, clear_hi;       // rows [clear_lo, clear_hi) of V's tile clear_j are no keys of the sequence
  int more;                              // 0: no work is left, the other fields are not set
  __device__ bool has(int t) const { return jhi[t] > jlo[t]; }
  __device__ bool active(int t, int j) const { return j >= jlo[t] && j < jhi[t]; }
  __device__ int top() const { return max(jhi[0], jhi[1]); }
  __device__ int bottom() const { return min(has(0) ? jlo[0] : 0x7fffffff, has(1) ? jlo[1] : 0x7fffffff); }
};

// Tiles of the sequences in order, the last tiles (the most keys) of each first. One warp; false:
// no such tile. With `check_all`, sequences past the tile are looked at too, for their bounds.
__device__ __forceinline__ bool find_job(const PromptParams& p, int64_t id, bool check_all, Job& job) {
  const int lane = threadIdx.x & 31, tpc = 2 * p.tt;
  const int64_t tile = id / p.heads_kv;
  int64_t before = 0;
  bool found = false;
  job.h = (int)(id % p.heads_kv);
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
  const int top = job.i0 + job.n + job.off;              // past the last position, at most lk
  const int bottom = p.window > 0 ? max(job.i0 + job.off - p.window + 1, 0) : 0;
  job.kbase = 0;
  if (p.window > 0 && top > 0) job.kbase = top - ((top - bottom + kKeys - 1) / kKeys) * kKeys;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = min(p.tt, job.n - t * p.tt), first = job.i0 + t * p.tt + job.off;   // first position
    const int hi = first + n;                                                         // past the last position
    job.jlo[t] = job.jhi[t] = 0;
    if (n > 0 && hi > 0) {
      job.jhi[t] = (hi - job.kbase + kKeys - 1) / kKeys;
      job.jlo[t] = p.window > 0 ? (max(first - p.window + 1, 0) - job.kbase) / kKeys : 0;
    }
  }
  // the one tile that reaches past the sequence: the lowest with a negative kbase, else the top one
  job.clear_j = -1;
  job.clear_lo = job.clear_hi = 0;
  if (job.top() > 0) {
    const int end = job.kbase + job.top() * kKeys;
    if (job.kbase < 0) {
      job.clear_j = 0;
      job.clear_hi = -job.kbase;
    } else if (end > job.lk) {
      job.clear_j = job.top() - 1;
      job.clear_lo = kKeys - (end - job.lk);
      job.clear_hi = kKeys;
    }
  }
  job.more = 1;
  return true;
}

constexpr int kJobSlots = 2;

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
  using L = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Job s_job[kJobSlots];
  __shared__ __align__(16) uint4 s_answer;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bars[21 + 2 * kJobSlots + 2 * L::kStages];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base + L::kOffQ, sKv = base + L::kOffKv;
  // mbarriers, one for each query tile: Q of a job loaded / read by its last product, O read, every
  // product done; two for each query tile, for key tiles in turn: S computed, P written, P V added to
  // O (one barrier for all key tiles would not do: the softmax may be two of them ahead of P V, and a
  // parity cannot tell that). Then the launcher's answer, the jobs and the ring of K and V
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t q_full = bars, q_empty = bars + 16, o_empty = bars + 32, drain = bars + 48, s_full = bars + 64,
                 p_full = bars + 96, o_full = bars + 128, answered = bars + 160, job_full = bars + 168,
                 job_empty = job_full + 8 * kJobSlots, kv_full = job_empty + 8 * kJobSlots,
                 kv_empty = kv_full + 8 * L::kStages;
  static_assert(168 + 16 * kJobSlots + 16 * L::kStages <= sizeof(s_bars), "barriers");

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), 512);
  if (tid == 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + 8 * t, 1);
      mbar_init(q_empty + 8 * t, 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full + 16 * t + 8 * b, 1);
        mbar_init(p_full + 16 * t + 8 * b, 4);
        mbar_init(o_full + 16 * t + 8 * b, 1);
      }
      mbar_init(o_empty + 8 * t, 4);
      mbar_init(drain + 8 * t, 1);
    }
    mbar_init(answered, 1);
    for (int s = 0; s < kJobSlots; ++s) {
      mbar_init(job_full + 8 * s, 1);
      mbar_init(job_empty + 8 * s, kSoftWarps + 3);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 2);      // both tiles' products
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
  griddep_wait();
  griddep_launch_dependents();
  bool ok = true;

  // Job `it` of this CTA, by one warp: waits for it; free_job frees its slot, once it has been read.
  auto wait_job = [&](int it) {
    const int s = it % kJobSlots;
    ok = wait_bar(job_full + 8 * s, (it / kJobSlots) & 1, p.wait_ns) && ok;
    ok = __all_sync(0xffffffffu, ok);
    return ok && s_job[s].more != 0;
  };
  auto free_job = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(job_empty + 8 * (it % kJobSlots));
  };
  auto take_job = [&](int it, Job& job) {
    if (!wait_job(it)) return false;
    job = s_job[it % kJobSlots];
    free_job(it);
    return true;
  };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loads
      // The ring holds K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1), tiles counted from the top: the
      // products of S run a key tile ahead of those with V.
      int n_q[2] = {0, 0}, c = 0;        // queries loaded; tiles of the ring loaded
      auto load_kv = [&](const Job& job, int j, const CUtensorMap* map) {
        const int s = c % L::kStages;
        ok = ok && wait_bar(kv_empty + 8 * s, ((c / L::kStages) & 1) ^ 1, p.wait_ns);
        if (!ok) return;
        mbar_arrive_expect_tx(kv_full + 8 * s, L::kKvBytes);
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          tma_3d(sKv + s * L::kKvBytes + d * kBlockK, map, 64 * d, job.h, job.k0 + job.kbase + kKeys * j, kv_full + 8 * s);
        ++c;
      };
      auto load_q = [&](const Job& job, int t) {
        ok = ok && wait_bar(q_empty + 8 * t, (n_q[t] & 1) ^ 1, p.wait_ns);
        if (!ok) return;
        mbar_arrive_expect_tx(q_full + 8 * t, (D / 64) * (uint32_t)(p.tt * p.group) * 128u);
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          tma_4d(sQ + t * L::kQBytes + d * kBlockQ, &p.qm, 64 * d, 0, job.h, job.q0 + job.i0 + t * p.tt, q_full + 8 * t);
        ++n_q[t];
      };
      Job job;
      for (int it = 0; take_job(it, job); ++it) {
        if (lane == 0) {
          const int top = job.top(), bottom = job.bottom();
          if (top > 0) load_kv(job, top - 1, &p.km);
          if (job.has(0)) load_q(job, 0);
          if (job.has(1)) load_q(job, 1);
          for (int j = top - 1; j >= bottom && ok; --j) {
            if (j > bottom) load_kv(job, j - 1, &p.km);
            load_kv(job, j, &p.vm);
          }
        }
        __syncwarp();
      }
      // nothing of this CTA's may be in flight when it ends, whatever the other roles did
      if (lane == 0) {
        for (int e = max(0, c - L::kStages); e < c; ++e)
          ok = wait_bar(kv_full + 8 * (e % L::kStages), (e / L::kStages) & 1, p.wait_ns) && ok;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (n_q[t]) ok = wait_bar(q_full + 8 * t, (n_q[t] - 1) & 1, p.wait_ns) && ok;
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // -------------------------------------------------------------- products of one query tile
      const int t = warp - kMmaWarp;
      const uint32_t tS = tmem + 128 * t, tO = tmem + 256 + 128 * t;
      const uint32_t id_qk = idesc_f16(kTile, kKeys, false, false, BF16), id_pv = idesc_f16(kTile, D, false, true, BF16);
      const uint64_t dq = sdesc(sQ + t * L::kQBytes, 16u, 1024u);
      auto wait = [&](uint32_t bar, int n) {
        ok = wait_bar(bar, n & 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return ok;
      };
      int n_q = 0, n_s = 0, n_p = 0, c = 0;      // jobs with keys for this tile, key tiles of S and P, tiles of the ring
      auto wait_kv = [&]() { return wait(kv_full + 8 * (c % L::kStages), c / L::kStages); };
      const uint32_t one = elect_one();
      auto free_kv = [&]() {
        umma_commit_one(one, kv_empty + 8 * (c % L::kStages));
        ++c;
      };
      // S of the next key tile, into the buffer whose P the product with V before last has read
      auto qk = [&](bool last) {
        const uint64_t dk = sdesc(sKv + (c % L::kStages) * L::kKvBytes, 16u, 1024u);
        const uint32_t at = tS + 64 * (n_s & 1);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss(one, at, dq + (((k >> 2) * kBlockQ + (k & 3) * 32u) >> 4), dk + (((k >> 2) * kBlockK + (k & 3) * 32u) >> 4), id_qk,
                  k > 0);
        umma_commit_one(one, s_full + 16 * t + 8 * (n_s & 1));
        if (last) umma_commit_one(one, q_empty + 8 * t);
        ++n_s;
      };
      auto pv = [&](bool acc) {
        const uint64_t dv = sdesc(sKv + (c % L::kStages) * L::kKvBytes, kBlockK, 1024u);
        const uint32_t at = tS + 64 * (n_p & 1);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) umma_ts(one, tO, at + 8 * k, dv + ((k * 16u * 128u) >> 4), id_pv, acc || k > 0);
        umma_commit_one(one, o_full + 16 * t + 8 * (n_p & 1));
        ++n_p;
      };
      Job job;
      for (int it = 0; take_job(it, job); ++it) {
        const int top = uniform(job.top()), bottom = uniform(job.bottom()), clear_j = uniform(job.clear_j);
        const int jlo = uniform(t ? job.jlo[1] : job.jlo[0]), jhi = uniform(t ? job.jhi[1] : job.jhi[0]);
        if (top == 0) continue;
        const bool has = jhi > jlo;
        if (has && !wait(q_full + 8 * t, n_q)) break;
        if (!wait_kv()) break;
        if (top == jhi) qk(top - 1 == jlo);
        free_kv();
        for (int j = top - 1; j >= bottom && ok; --j) {
          if (j > bottom) {
            if (!wait_kv()) break;
            if (j - 1 >= jlo && j - 1 < jhi) qk(j - 1 == jlo);
            free_kv();
          }
          if (!wait_kv()) break;
          if (j >= jlo && j < jhi) {
            if (j == clear_j) {          // rows that are no keys of the sequence (both warps write the same zeros)
              const uint32_t v = sKv + (c % L::kStages) * L::kKvBytes;
              for (int x = job.clear_lo * 8 + lane; x < job.clear_hi * 8; x += 32)
#pragma unroll
                for (int d = 0; d < D / 64; ++d) sts128(v + d * kBlockK + x * 16u, 0u, 0u, 0u, 0u);
              fence_async_smem();
              __syncwarp();
            }
            // the first product of a job overwrites O: the last job's must have been read
            if (j == jhi - 1 && !wait(o_empty + 8 * t, n_q ^ 1)) break;
            if (!wait(p_full + 16 * t + 8 * (n_p & 1), n_p >> 1)) break;
            pv(j < jhi - 1);
          }
          free_kv();
        }
        if (!ok) break;
        n_q += has;
      }
      umma_commit_one(one, drain + 8 * t);       // every product is done before the tensor memory is freed
      ok = wait_bar(drain + 8 * t, 0, p.wait_ns) && ok;
    } else {
      // -------------------------------------------------------------- what comes next
      // A block is taken only when the work before the last has been done by every role, so that no CTA
      // holds back more than one piece of work (taking three ahead left ragged batches uneven).
      const uint32_t answer = smem_u32(&s_answer);
      uint32_t block = blockIdx.x;
      int it = 0;
      auto wait_slot = [&]() {
        ok = wait_bar(job_empty + 8 * (it % kJobSlots), ((it / kJobSlots) & 1) ^ 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      for (int n = 0; ok; ++n) {
        Job job;
        if (find_job(p, block, block == gridDim.x - 1, job)) {
          if (!wait_slot()) break;
          if (lane == 0) {
            s_job[it % kJobSlots] = job;
            mbar_arrive(job_full + 8 * (it % kJobSlots));
          }
          ++it;
        }
        if (!wait_slot()) break;
        if (lane == 0) {
          fence_async_smem();            // the last answer has been read
          mbar_arrive_expect_tx(answered, 16);
          next_block_ask(answer, answered);
        }
        __syncwarp();
        ok = wait_bar(answered, n & 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool more = next_block_take(answer, block);
        __syncwarp();
        if (!more) {
          if (lane == 0) {
            s_job[it % kJobSlots].more = 0;
            mbar_arrive(job_full + 8 * (it % kJobSlots));
          }
          break;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax: one row per thread
    // Shared memory is busy with the products' operands, so this loop keeps out of it: no exchange
    // between warps (two warps per row, half the keys each, took 1.5 times as long), no spilled
    // registers. What the epilogue needs of the job is read again there, and the values that follow
    // from it are not kept across the loop.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = warp >> 2;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * t, tO = tS + 256u;
    const float scale = p.scale_log2;
    int n_s = 0;                         // key tiles so far
    for (int it = 0; wait_job(it); ++it) {
      int j, jlo, hi, lo, whole_hi, whole_lo;
      {
        const Job& job = s_job[it % kJobSlots];
        const int r = (warp & 3) * 32 + lane, r_tok = t * p.tt + r / p.group;
        const int first = job.i0 + job.off - job.kbase;                // the first token's position, from kbase on
        const int floor = -job.kbase;                                  // key 0 (kbase < 0: with a window)
        const bool real = r < p.tt * p.group && r_tok < job.n;
        jlo = t ? job.jlo[1] : job.jlo[0];
        j = (t ? job.jhi[1] : job.jhi[0]) - 1;
        // this row's keys, and those that every row of the tile sees, from tile j's first key on
        hi = (real ? max(first + r_tok + 1, 0) : 0) - kKeys * j;
        lo = (real && p.window > 0 ? max(first + r_tok - p.window + 1, floor) : 0) - kKeys * j;
        whole_hi = first + t * p.tt + 1 - kKeys * j;
        whole_lo = (p.window > 0 ? max(first + min(job.n, (t + 1) * p.tt) - p.window, floor) : 0) - kKeys * j;
      }
      float m = -INFINITY, l = 0.f;
      bool later = false;                // a tile of this job has gone into O
      const bool keys = j >= jlo;
      for (; j >= jlo; --j, ++n_s) {
        ok = wait_bar(s_full + 16 * t + 8 * (n_s & 1), (n_s >> 1) & 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        softmax_tile<D, BF16>(
            tS + 64 * (n_s & 1), tO, hi > 0, scale, m, l, later,
            [&](uint32_t(&s)[2][32]) {
              if (kKeys > whole_hi || 0 < whole_lo) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c)
                  if (c >= hi || c < lo) s[c >> 5][c & 31] = 0xFF800000u;   // -inf
              }
            },
            [&]() {                      // the last tile's P V is in O
              ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, p.wait_ns) && ok;
              tc_fence_after();
            });
        later = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * (n_s & 1));
        hi += kKeys;
        lo += kKeys;
        whole_hi += kKeys;
        whole_lo += kKeys;
      }
      if (!ok) break;
      // -------------------------------------------------------------- O / l
      if (keys) {
        ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, p.wait_ns) && ok;   // the last P V
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const Job& job = s_job[it % kJobSlots];
      int group = p.group;               // opaque: what follows from it is computed here, not before the loop
      asm volatile("" : "+r"(group));
      const uint32_t stage = base + L::kOffStage + (uint32_t)warp * 2048u;
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const int64_t row0 = (int64_t)job.q0 + job.i0;
      uint16_t* dst[4];                  // where this lane writes its piece of rows 8 i + lane / 4; NULL: no such row
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = (warp & 3) * 32 + 8 * i + (lane >> 2), tok = t * p.tt + rr / group;
        dst[i] = rr < p.tt * group && tok < job.n
                     ? p.out + (row0 + tok) * p.out_stride + (int64_t)(job.h * group + rr % group) * D + 8 * (lane & 3)
                     : nullptr;
      }
      if (p.lse) {
        const int r = (warp & 3) * 32 + lane, tok = t * p.tt + r / group;
        if (r < p.tt * group && tok < job.n)
          p.lse[(row0 + tok) * p.heads_q + job.h * group + r % group] = l != 0.f ? (m * scale + log2f(l)) * kLn2 : -INFINITY;
      }
      free_job(it);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (keys) {
          TMEM_LD32(tO + 32 * c, o);
          tmem_wait_ld();
          tmem_regs_ready(o);
          if (c == D / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty + 8 * t);
          }
        }
        // through shared memory, so that four lanes write 64 bytes of a row together
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t y[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float a = l != 0.f ? __uint_as_float(o[8 * e + 2 * u]) * inv : 0.f;
            const float b = l != 0.f ? __uint_as_float(o[8 * e + 2 * u + 1]) * inv : 0.f;
            y[u] = pack2<BF16>(a, b);
          }
          sts128(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 8 * i + (lane >> 2);
          const uint4 y = lds128(stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
          if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + 32 * c) = y;
        }
        __syncwarp();
      }
    }
  }
  if (!ok) flag_status(p.status, HSA_FLAG_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int D, bool BF16>
cudaError_t launch(const PromptParams& p, unsigned blocks, cudaStream_t s) {
  auto kernel = prompt_attn_kernel<D, BF16>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), Shape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), Shape<D>::kSmem, s, p);
}

}  // namespace

TensorMapEncoder tensor_map_encoder() {
  static const TensorMapEncoder fn = []() -> TensorMapEncoder {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<TensorMapEncoder>(f);
  }();
  return fn;
}

cudaError_t launch_prompt_attn(const hsa_prompt_args& a, uint32_t* status, uint64_t wait_ns, cudaStream_t s) {
  const TensorMapEncoder encode = tensor_map_encoder();
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
  p.scale_log2 = a.sm_scale * kLog2e;
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
    // k and v as [row][key-value head][dim]: a box is 64 rows x 64 dims. Without any rows the maps
    // are never used (no sequence has keys); they stand on q then.
    const cuuint64_t dims[3] = {d, (cuuint64_t)p.heads_kv, (cuuint64_t)(a.n_k > 0 ? a.n_k : 1)};
    const cuuint64_t strides[2] = {2 * d, 2 * (cuuint64_t)(i ? a.v_stride : a.k_stride)};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kKeys};
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
