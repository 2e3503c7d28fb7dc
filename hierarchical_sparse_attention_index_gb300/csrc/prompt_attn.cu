// Causal attention over packed prompts with grouped heads (hsa_prompt_attn):
//   o_i = sum_j softmax_j(scale q_i.k_j) v_j over the keys j a query sees.
//
// Bound: the two products, 4 d flops per visible (query, key) pair and head, on the tensor cores;
// the exponentials and the rest of the softmax run beside them. One CTA per SM takes two tiles of
// 128 rows at a time. A row is one query head of one token: the `group` heads that share a key-value
// head stand together (tt = 128 / group tokens per tile), so that grouped heads share every key tile
// and a tile spans few tokens, which keeps the masked part at the diagonal small.
//  - CTAs stay and take the next block's work themselves (cluster launch control), while the loads
//    of the next work already run; the work with the most keys comes first;
//  - one warp loads Q, and 64-key tiles of K and V into a ring, by TMA (128-byte swizzle);
//  - a warp per query tile issues its tcgen05 products: S = Q K^T (128 x 64, fp32 in tensor memory,
//    two buffers, one key tile ahead), then O += P V with P read from tensor memory and V as an
//    MN-major operand. So S of the next key tile is there when the softmax comes to it. (A product
//    for 64 keys reads 6 KB of shared memory in the 32 clocks that it computes, 128 bytes a clock
//    can be read; one for 128 keys reads 8 KB in 64, but leaves room for one buffer only: 16,384
//    tokens took the same time, packed prompts 15 % more);
//  - a warp group does the softmax of each tile, one row per thread (no shuffles): the running
//    maximum and sum in fp32, P rounded to the operand type (off by at most a relative 2^-8 in bf16, in f16 2^-11 down
//    to 2^-21 of a row's largest weight and 2^-32 of it below, independent from key to key) over S's columns. The maximum is only
//    raised, and O rescaled in tensor memory, when a logit passes it by 2^8: weights stay below 256 (2^15 in f16), and after the first
//    tiles that hardly happens, so the rescaling needs no warps of its own;
//  - four warps write the results, while the softmax is at the next work (in a window of 128 the writing
//    took as long as half of the softmax);
//  - keys come from the diagonal downwards, so the first tile already holds each row's own key;
//  - the rows of V's tiles that are no keys of the sequence are cleared before use: their weights
//    are zero, but zero times another sequence's infinity would not be.
// TMEM: S 2 x 64 columns per query tile (P over the first half of its buffer), O head_dim columns each.
// Every wait is bounded; a role that gives up leaves its loop, and the others follow at their next
// wait.
// Measured: 16,384 tokens, 32 heads over 4, 128 dims 1,360-1,440 us, 1,530-1,620 TFLOP/s, 0.79-0.83 of the measured bf16
// peak (1,463-1,481 under the power cap); without the softmax's part 1,340 us, where shared memory bounds the products. 12
// packed prompts, 64 heads over 8, 365 us, 0.70 (395-404 under the cap); a window of 128 over 32,768 tokens of 64 dims 177 us. With 64 dims a key tile takes
// 1,200 clocks, of which the softmax's chain (logits, maximum, exponentials, P) is 1,000 and the exponentials alone are 512.
#include "hsa_flash.cuh"
#include "hsa_dense.h"

namespace hsa {
namespace {

constexpr int kTile = 128;               // rows of a query tile
constexpr int kKeys = 64;                // keys of a key tile
constexpr int kSoftWarps = 8;            // 4 per query tile: warp groups 0 and 1
constexpr int kMmaWarp = 8, kLoadWarp = 10;              // a warp per query tile's products; warp 11 finds the work
constexpr int kOutWarp = 12;             // warps 12..15 write the results
constexpr int kThreads = 16 * 32;
// registers per thread: 128 at launch (65,536 over 512 threads), then 152 for the softmax groups, whose
// threads hold a row of 64 logits, and 104 for the other two: 2 x 152 + 2 x 104 = 4 x 128
constexpr int kLaunchRegs = 128, kSoftRegs = 152, kOtherRegs = 104;
static_assert(2 * kSoftRegs + 2 * kOtherRegs <= 4 * kLaunchRegs, "setmaxnreg draws on the launch's registers");
constexpr int kSeqs = 512;               // batches up to this are held in shared memory and worked off by size
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
  int32_t wide;                          // rows of out start on 32-byte boundaries
  uint32_t* status;
  uint64_t wait_ns;
};

template <int D>
struct Shape {
  static constexpr uint32_t kQBytes = (D / 64) * kBlockQ, kKvBytes = (D / 64) * kBlockK;
  static constexpr int kStages = 8;                              // tiles of K and V in the ring
  static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kQBytes, kOffSeq = kOffKv + kStages * kKvBytes, kSmem = kOffSeq + kSeqs * 24 + 1024;   // + alignment slack
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
  __device__ int top() const { return max(jhi[0], jhi[1]); }
  __device__ int bottom() const { return min(has(0) ? jlo[0] : 0x7fffffff, has(1) ? jlo[1] : 0x7fffffff); }
};

struct Seq {
  int q0, lq, k0, lk;
  int count, base;                       // pieces of work, and the level of the first
};
// Sequence b, empty if its own bounds are bad
__device__ __forceinline__ Seq load_seq(const PromptParams& p, int b, bool& good) {
  Seq s = {};
  good = true;
  if (b < p.batch) {
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    good = q0 >= 0 && q0 <= q1 && q1 <= p.n_q && k0 >= 0 && k0 <= k1 && k1 <= p.n_k;
    if (good)
      s = Seq{q0, q1 - q0, k0, k1 - k0};
    else
      flag_status(p.status, HSA_FLAG_INDEX_RANGE);
  }
  const int tpc = 2 * p.tt;
  s.count = (s.lq + tpc - 1) / tpc;
  s.base = p.window > 0 ? 0 : max(0, s.lk - s.lq) / tpc;
  return s;
}
// Sequences first + lane, by one warp; one that starts before an earlier one ends is empty too, so that no row
// has two and the pieces are no more than prompt_blocks counts. `high`: where the earlier ones end. Bounds that ascend
// ask for one comparison; behind a bad one each lane needs the ends of those before it.
__device__ __forceinline__ Seq load_seqs(const PromptParams& p, int first, int& high) {
  const int lane = threadIdx.x & 31;
  bool good;
  Seq s = load_seq(p, first + lane, good);
  const int end = s.lq > 0 ? s.q0 + s.lq : 0;
  int before = high;
  if (__any_sync(0xffffffffu, !good)) {
    int upto = end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = max(upto, y);
    }
    upto = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane > 0) before = max(before, upto);
  }
  high = max(high, __reduce_max_sync(0xffffffffu, end));
  if (s.lq > 0 && s.q0 < before) {
    flag_status(p.status, HSA_FLAG_INDEX_RANGE);
    s.lq = s.count = 0;
  }
  return s;
}

// The order of the work. Every 2 tt tokens of a sequence are one piece; the pieces with the most keys
// come first, so that the last ones to be taken are short. Sequence b's pieces have the levels base_b ..
// base_b + count_b - 1 (a level is about 2 tt keys); those of one level stand in the order of the
// sequences. One warp; the sequences lie in shared memory.
struct Order {
  static constexpr int kHeld = 4;        // up to 128 sequences' counts and levels stay in registers: shared memory
  const Seq* seq;                        // answers slowly beside the products (6,000 clocks a search, 1,000 so)
  int batch, total, levels;              // pieces in all; levels are 0 .. levels - 1
  int count[kHeld], base[kHeld];         // of sequences lane + 32 k
  __device__ void hold(const Seq* s, int n) {
    const int lane = threadIdx.x & 31;
    seq = s;
    batch = n;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int b = lane + 32 * k;
      count[k] = b < n ? s[b].count : 0;
      base[k] = b < n ? s[b].base : 0;
    }
    total = above(0);
    int top = 0;
    for (int b = lane; b < n; b += 32) top = max(top, s[b].base + s[b].count);
    levels = __reduce_max_sync(0xffffffffu, top);
  }
  // pieces of level x and above
  __device__ int above(int x) const {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) n += max(0, count[k] - max(0, x - base[k]));
    for (int b = (threadIdx.x & 31) + 32 * kHeld; b < batch; b += 32) n += max(0, seq[b].count - max(0, x - seq[b].base));
    return __reduce_add_sync(0xffffffffu, n);
  }
  // piece number r: the sequence, and which of its pieces
  __device__ bool find(int r, int& which, int& i) const {
    if (r >= total) return false;
    which = 0;
    i = total - 1 - r;
    if (batch == 1) return true;
    int x = 0, past = levels;            // above(x) > r >= above(past)
    while (past - x > 1) {
      const int mid = (x + past) >> 1;
      if (above(mid) > r) x = mid; else past = mid;
    }
    int left = r - above(x + 1);
    auto among = [&](int first, int c, int b) {          // of 32 sequences from `first`, this lane's with c pieces from level b on
      uint32_t m = __ballot_sync(0xffffffffu, b <= x && x < b + c);
      if (left >= __popc(m)) {
        left -= __popc(m);
        return false;
      }
      for (; left > 0; --left) m &= m - 1;
      which = __ffs(m) - 1;
      i = x - __shfl_sync(0xffffffffu, b, which);
      which += first;
      return true;
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (32 * k < batch && among(32 * k, count[k], base[k])) return true;
    for (int first = 32 * kHeld; first < batch; first += 32) {
      const int b = first + (threadIdx.x & 31);
      if (among(first, b < batch ? seq[b].count : 0, b < batch ? seq[b].base : 0)) return true;
    }
    return false;
  }
};

// Larger batches are worked off in the order of the sequences, the last piece of each first. A search starts
// at the 32 sequences where the last one ended (`first`, with `before` pieces before them, which end at `high`): a CTA's
// blocks come in rising order, so all its searches together pass over the batch about once.
__device__ __forceinline__ bool find_in_turn(const PromptParams& p, int r, Seq& out, int& i, int& first, int& before, int& high) {
  const int lane = threadIdx.x & 31;
  if (r < before) first = before = high = 0;
  for (; first < p.batch; first += 32) {
    int end = high;
    const Seq s = load_seqs(p, first, end);
    int upto = s.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    upto += before;
    const uint32_t past = __ballot_sync(0xffffffffu, upto > r);
    if (past) {
      const int src = __ffs(past) - 1;
      out.q0 = __shfl_sync(0xffffffffu, s.q0, src);
      out.lq = __shfl_sync(0xffffffffu, s.lq, src);
      out.k0 = __shfl_sync(0xffffffffu, s.k0, src);
      out.lk = __shfl_sync(0xffffffffu, s.lk, src);
      i = __shfl_sync(0xffffffffu, upto, src) - 1 - r;
      return true;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
    high = end;
  }
  return false;
}

__device__ __forceinline__ void make_job(const PromptParams& p, const Seq& s, int i, int h, Job& job) {
  const int tpc = 2 * p.tt;
  job.h = h;
  job.q0 = s.q0;
  job.k0 = s.k0;
  job.lk = s.lk;
  job.i0 = i * tpc;
  job.n = min(tpc, s.lq - job.i0);
  job.off = s.lk - s.lq;
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
}

constexpr int kJobSlots = 4;
constexpr int kAhead = 8;                // key tiles left to load when the next piece of work is looked for

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
  using L = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Job s_job[kJobSlots];
  __shared__ __align__(16) uint4 s_answer;
  __shared__ uint32_t s_tmem;
  __shared__ uint16_t s_tok[kTile], s_head[kTile];       // of a query tile's rows; token 0xFFFF: no row
  __shared__ float2 s_ml[2][kTile];                      // each query tile's (maximum, sum)
  __shared__ __align__(8) uint64_t s_bars[23 + 3 * kJobSlots + 2 * L::kStages];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base + L::kOffQ, sKv = base + L::kOffKv;
  // mbarriers, one for each query tile: Q of a job loaded / read by its last product, O and (m, l) read,
  // every product done, (m, l) written; two for each query tile, for key tiles in turn: S computed, P written, P V added to
  // O (one barrier for all key tiles would not do: the softmax may be two of them ahead of P V, and a
  // parity cannot tell that). Then the launcher's answer, the jobs (posted, done, loads issued) and the ring of K and V
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t q_full = bars, q_empty = bars + 16, o_empty = bars + 32, drain = bars + 48, s_full = bars + 64,
                 p_full = bars + 96, o_full = bars + 128, ml_full = bars + 160, answered = bars + 176, job_full = bars + 184,
                 job_empty = job_full + 8 * kJobSlots, job_loaded = job_empty + 8 * kJobSlots, kv_full = job_loaded + 8 * kJobSlots,
                 kv_empty = kv_full + 8 * L::kStages;
  static_assert(184 + 24 * kJobSlots + 16 * L::kStages <= sizeof(s_bars), "barriers");

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
      mbar_init(ml_full + 8 * t, 4);
      mbar_init(drain + 8 * t, 1);
    }
    mbar_init(answered, 1);
    for (int s = 0; s < kJobSlots; ++s) {
      mbar_init(job_full + 8 * s, 1);
      mbar_init(job_loaded + 8 * s, 1);
      mbar_init(job_empty + 8 * s, kSoftWarps + 3 + 4);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 2);      // both tiles' products
    }
    fence_mbar_init();
  }
  if (tid < kTile) {
    s_tok[tid] = tid < p.tt * p.group ? tid / p.group : 0xFFFF;
    s_head[tid] = tid % p.group;
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

  if (warp >= kSoftWarps && warp < kOutWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loads
      // The ring holds K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1), tiles counted from the top: the
      // products of S run a key tile ahead of those with V.
      int n_q[2] = {0, 0}, c = 0;        // queries loaded; tiles of the ring loaded
      const uint32_t one = elect_one();
      auto wait = [&](uint32_t bar, int n) {
        ok = wait_bar(bar, n & 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      auto load_kv = [&](int h, int row, const CUtensorMap* map) {
        const int s = c % L::kStages;
        if (!wait(kv_empty + 8 * s, (c / L::kStages) ^ 1)) return;
        if (one) mbar_arrive_expect_tx(kv_full + 8 * s, L::kKvBytes);
        __syncwarp();
#pragma unroll
        for (int d = 0; d < D / 64; ++d) tma_3d_one(one, sKv + s * L::kKvBytes + d * kBlockK, map, 64 * d, h, row, kv_full + 8 * s);
        ++c;
      };
      auto load_q = [&](int h, int row, int t) {
        if (!ok || !wait(q_empty + 8 * t, n_q[t] ^ 1)) return;
        if (one) mbar_arrive_expect_tx(q_full + 8 * t, (D / 64) * (uint32_t)(p.tt * p.group) * 128u);
        __syncwarp();
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          tma_4d_one(one, sQ + t * L::kQBytes + d * kBlockQ, &p.qm, 64 * d, 0, h, row, q_full + 8 * t);
        ++n_q[t];
      };
      Job job;
      for (int it = 0; take_job(it, job); ++it) {
        const int top = uniform(job.top()), bottom = uniform(job.bottom()), ask = min(top - 1, bottom + kAhead);
        const int h = uniform(job.h), row = uniform(job.k0 + job.kbase), q_row = uniform(job.q0 + job.i0);
        if (top == 0 && lane == 0) mbar_arrive(job_loaded + 8 * (it % kJobSlots));
        if (top > 0) load_kv(h, row + kKeys * (top - 1), &p.km);
        if (job.has(0)) load_q(h, q_row, 0);
        if (job.has(1)) load_q(h, q_row + p.tt, 1);
        for (int j = top - 1; j >= bottom && ok; --j) {
          if (j == ask && lane == 0) mbar_arrive(job_loaded + 8 * (it % kJobSlots));
          if (j > bottom) load_kv(h, row + kKeys * (j - 1), &p.km);
          if (ok) load_kv(h, row + kKeys * j, &p.vm);
        }
        if (!ok) break;
      }
      // nothing of this CTA's may be in flight when it ends, whatever the other roles did
      if (lane == 0) {
        for (int e = max(0, c - L::kStages); e < c; ++e)
          ok = drain_bar(kv_full + 8 * (e % L::kStages), (e / L::kStages) & 1) && ok;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (n_q[t]) ok = drain_bar(q_full + 8 * t, (n_q[t] - 1) & 1) && ok;
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
      // A job as this warp needs it
      struct Mine {
        int top, bottom, jlo, jhi, clear_j, clear_lo, clear_hi;
      };
      auto mine_of = [&](const Job& job) {
        return Mine{uniform(job.top()), uniform(job.bottom()), uniform(t ? job.jlo[1] : job.jlo[0]), uniform(t ? job.jhi[1] : job.jhi[0]),
                    uniform(job.clear_j), uniform(job.clear_lo), uniform(job.clear_hi)};
      };
      auto ready = [&](uint32_t bar, int n) { return __all_sync(0xffffffffu, mbar_test(bar, n & 1)); };
      // The first S of the next job is computed before the last P V of this one where it can be, so that the
      // softmax finds it when it comes there: `taken`, the next job is known; `begun`, its first S is issued.
      bool taken = false, begun = false;
      Mine next = {};
      for (int it = 0;; ++it) {
        Mine job = next;
        if (!taken) {
          if (!wait_job(it)) break;
          job = mine_of(s_job[it % kJobSlots]);
          free_job(it);
        }
        taken = false;
        if (job.top == 0) continue;
        const bool has = job.jhi > job.jlo;
        if (!begun) {
          if (has && !wait(q_full + 8 * t, n_q)) break;
          if (!wait_kv()) break;
          if (job.top == job.jhi) qk(job.top - 1 == job.jlo);
          free_kv();
        }
        begun = false;
        for (int j = job.top - 1; j >= job.bottom && ok; --j) {
          if (j > job.bottom) {
            if (!wait_kv()) break;
            if (j - 1 >= job.jlo && j - 1 < job.jhi) qk(j - 1 == job.jlo);
            free_kv();
          } else if (ready(job_full + 8 * ((it + 1) % kJobSlots), (it + 1) / kJobSlots) && s_job[(it + 1) % kJobSlots].more) {
            next = mine_of(s_job[(it + 1) % kJobSlots]);
            free_job(it + 1);
            taken = true;
            const int q = n_q + has, k = c + 1;          // V of this tile comes first in the ring
            if (next.top > 0 && (next.jhi == next.jlo || ready(q_full + 8 * t, q)) &&
                ready(kv_full + 8 * (k % L::kStages), k / L::kStages)) {
              tc_fence_after();
              const int v = c;
              c = k;
              if (next.top == next.jhi) qk(next.top - 1 == next.jlo);
              free_kv();
              c = v;
              begun = true;
            }
          }
          if (!wait_kv()) break;
          if (j >= job.jlo && j < job.jhi) {
            if (j == job.clear_j) {      // rows that are no keys of the sequence (both warps write the same zeros)
              const uint32_t v = sKv + (c % L::kStages) * L::kKvBytes;
              for (int x = job.clear_lo * 8 + lane; x < job.clear_hi * 8; x += 32)
#pragma unroll
                for (int d = 0; d < D / 64; ++d) sts128(v + d * kBlockK + x * 16u, 0u, 0u, 0u, 0u);
              fence_async_smem();
              __syncwarp();
            }
            // the first product of a job overwrites O: the last job's must have been read
            if (j == job.jhi - 1 && !wait(o_empty + 8 * t, n_q ^ 1)) break;
            if (!wait(p_full + 16 * t + 8 * (n_p & 1), n_p >> 1)) break;
            pv(j < job.jhi - 1);
          }
          free_kv();
        }
        if (!ok) break;
        c += begun;                      // the next job's first K
        n_q += has;
      }
      umma_commit_one(one, drain + 8 * t);       // every product is done before the tensor memory is freed
      ok = drain_bar(drain + 8 * t, 0) && ok;
    } else {
      // -------------------------------------------------------------- what comes next
      // The next block is taken when few of this piece's key tiles are left to load: a CTA that held more
      // would leave others without (taking a piece ahead from the start made a batch of chunks, two
      // pieces for each SM, last 1.4 times its share), one that took it at the end would wait for it.
      // Short pieces are posted up to four ahead: finding and starting one takes longer than its loop.
      const uint32_t answer = smem_u32(&s_answer);
      uint32_t block = blockIdx.x;
      int it = 0;
      auto wait_slot = [&]() {
        ok = wait_bar(job_empty + 8 * (it % kJobSlots), ((it / kJobSlots) & 1) ^ 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      Seq* seqs = reinterpret_cast<Seq*>(smem_raw + (base - raw) + L::kOffSeq);
      Order order;
      if (p.batch <= kSeqs) {
        for (int first = 0, high = 0; first < p.batch; first += 32) {
          const Seq s = load_seqs(p, first, high);
          if (first + lane < p.batch) seqs[first + lane] = s;
        }
        __syncwarp();
        order.hold(seqs, p.batch);
      }
      bool is_long = false;
      int in_turn = 0, pieces = 0, high = 0;     // find_in_turn's place
      for (int n = 0; ok; ++n) {
        Job job;
        Seq seq;
        int which = 0, i = 0;
        const int h = (int)(block % (uint32_t)p.heads_kv), r = (int)(block / (uint32_t)p.heads_kv);
        bool found;
        if (p.batch <= kSeqs) {
          found = order.find(r, which, i);
          if (found) seq = seqs[which];
        } else {
          found = find_in_turn(p, r, seq, i, in_turn, pieces, high);
          bool good;
          if (block == gridDim.x - 1)    // every sequence's bounds are looked at once
            for (int b = lane; b < p.batch; b += 32) load_seq(p, b, good);
        }
        if (found) {
          make_job(p, seq, i, h, job);
          if (!wait_slot()) break;
          if (lane == 0) {
            s_job[it % kJobSlots] = job;
            mbar_arrive(job_full + 8 * (it % kJobSlots));
          }
          ++it;
          is_long = job.top() - job.bottom() > kAhead;
        }
        if (!wait_slot()) break;
        if (is_long) {
          ok = wait_bar(job_loaded + 8 * ((it - 1) % kJobSlots), ((it - 1) / kJobSlots) & 1, p.wait_ns) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (lane == 0) {
          fence_async_smem();            // the last answer has been read
          mbar_arrive_expect_tx(answered, 16);
          next_block_ask(answer, answered);
        }
        __syncwarp();
        ok = drain_bar(answered, n & 1) && ok;
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
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax: one row per thread
    // Shared memory is busy with the products' operands, so this loop keeps out of it: no exchange
    // between warps (two warps per row, half the keys each, took 1.5 times as long), no spilled registers.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * t, tO = tS + 256u;
    const float scale = p.scale_log2;
    int n_s = 0, n_o = 0;                // key tiles, and jobs with keys, so far
    for (int it = 0; wait_job(it); ++it) {
      int j, jlo, hi, lo, whole_hi, whole_lo;
      {
        const Job& job = s_job[it % kJobSlots];
        const int r_tok = t * p.tt + s_tok[r];
        const int first = job.i0 + job.off - job.kbase;                // the first token's position, from kbase on
        const int floor = -job.kbase;                                  // key 0 (kbase < 0: with a window)
        const bool real = s_tok[r] != 0xFFFF && r_tok < job.n;
        jlo = t ? job.jlo[1] : job.jlo[0];
        j = (t ? job.jhi[1] : job.jhi[0]) - 1;
        // this row's keys, and those that every row of the tile sees, from tile j's first key on
        hi = (real ? max(first + r_tok + 1, 0) : 0) - kKeys * j;
        lo = (real && p.window > 0 ? max(first + r_tok - p.window + 1, floor) : 0) - kKeys * j;
        whole_hi = first + t * p.tt + 1 - kKeys * j;
        whole_lo = (p.window > 0 ? max(first + min(job.n, (t + 1) * p.tt) - p.window, floor) : 0) - kKeys * j;
      }
      free_job(it);
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
              if (kKeys > whole_hi || 0 < whole_lo) mask_row(s, lo, hi);
            },
            [&]() {                      // the last tile's P V is in O
              ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, p.wait_ns) && ok;
              ok = __all_sync(0xffffffffu, ok);
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
      if (keys) {                        // (m, l) to the warps that write, when they have read the last job's
        ok = wait_bar(o_empty + 8 * t, (n_o & 1) ^ 1, p.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++n_o;
        s_ml[t][r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full + 8 * t);
      }
    }
  } else {
    // ---------------------------------------------------------------- O / l, while the softmax is at the next job
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // Each lane writes its row, 32 bytes at a time where the rows allow it: that takes more write
    // transactions than gathering rows in shared memory first, but shared memory is what is scarce here
    // (a window of 128 over 32,768 tokens took 214 us that way when it took 187 so).
    const int r = (warp & 3) * 32 + lane, tok = s_tok[r], head = s_head[r];
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int n_s[2] = {0, 0}, n_o[2] = {0, 0};
    Job job;
    for (int it = 0; ok && take_job(it, job); ++it) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tiles = job.jhi[t] - job.jlo[t];
        const bool mine = tok < job.n - t * p.tt;        // this lane has a row
        const int64_t row = (int64_t)job.q0 + job.i0 + t * p.tt + tok;
        const int hq = job.h * p.group + head;
        uint16_t* dst = p.out + row * p.out_stride + hq * D;
        float m = -INFINITY, l = 0.f;
        if (tiles > 0) {
          ok = ok && wait_bar(ml_full + 8 * t, n_o[t] & 1, p.wait_ns);
          n_s[t] += tiles;
          ++n_o[t];
          ok = ok && wait_bar(o_full + 16 * t + 8 * ((n_s[t] - 1) & 1), ((n_s[t] - 1) >> 1) & 1, p.wait_ns);   // the last P V
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const float2 ml = s_ml[t][r];
          m = ml.x;
          l = ml.y;
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32], y[16];
          if (tiles > 0) {
            TMEM_LD32(tmem + lanes + 256u + 128u * t + 32u * c, o);
            tmem_wait_ld();
            tmem_regs_ready(o);
            if (c == D / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(o_empty + 8 * t);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e] = pack2<BF16>(l != 0.f ? __uint_as_float(o[2 * e]) * inv : 0.f, l != 0.f ? __uint_as_float(o[2 * e + 1]) * inv : 0.f);
          if (mine) {
            if (p.wide) {
              st_global_256(dst + 32 * c, y);
              st_global_256(dst + 32 * c + 16, y + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(dst + 32 * c + 2 * e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
          }
        }
        if (p.lse && mine) p.lse[row * p.heads_q + hq] = l != 0.f ? (fmaf(m, p.scale_log2, -kLift<BF16>) + log2f(l)) * kLn2 : -INFINITY;
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
  static const bool fits = launches_with(kernel, kLaunchRegs);
  if (!fits) return cudaErrorInvalidConfiguration;
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

// At most n_q / (2 tt) whole pieces of 2 tt tokens and one more per sequence, and no more than tokens
int64_t prompt_blocks(const hsa_prompt_args& a) {
  return imin64(a.n_q / (2 * (kTile / (a.heads_q / a.heads_kv))) + a.batch, a.n_q + 1) * a.heads_kv;
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
  p.window = (int32_t)imin64(a.window, 1 << 28);         // beyond every sequence, and its differences fit 32 bits
  p.n_q = a.n_q;
  p.n_k = a.n_k;
  p.out_stride = a.out_stride;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k ? a.cu_k : a.cu_q;
  p.scale_log2 = a.sm_scale * kLog2e;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.wide = ((uintptr_t)a.out % 32 == 0 && a.out_stride % 16 == 0) ? 1 : 0;
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
  const int64_t blocks = prompt_blocks(a);
  if (a.head_dim == 128)
    return a.dtype == HSA_BF16 ? launch<128, true>(p, (unsigned)blocks, s) : launch<128, false>(p, (unsigned)blocks, s);
  return a.dtype == HSA_BF16 ? launch<64, true>(p, (unsigned)blocks, s) : launch<64, false>(p, (unsigned)blocks, s);
}

}  // namespace hsa
