// Attention of new tokens over a paged cache for many query rows per key-value head (several queries,
// large groups) and 16-bit pages, on tcgen05; paged_attn.cu has the form for few rows and for E4M3.
//   o = sum_j softmax_j(scale q.k_j) v_j over the positions j a query sees.
//
// Bound: the reads of the pages from HBM, as with few rows, as long as the products keep up. The
// warp MMA does not: its 8-column tiles of queries are issued and softmaxed by the same few warps, and
// past 32 rows the keys would be read again. Here up to 128 rows (queries x heads of the group) are one
// tile of a tcgen05 product, and a 64-key tile of 32 KB takes about 700 clocks, in which an SM's share
// of HBM brings half as much. The split of a CTA's job falls into two halves, one for each stream t:
// a ring of K and V tiles, a warp that issues the products, a warp group with a query row per thread
// for the softmax, buffers of S and an accumulator in tensor memory; the two streams fill each other's
// waits. A row without a query (35 rows fill 35 of 128) costs nothing but its lane: warps without any
// skip the softmax.
//  - one warp loads: K and V tiles as boxes of gcd(page size, 64) rows by TMA (128-byte swizzle), two
//    lanes and more issuing; rows past the visible length inside a box are cleared before use (zero
//    times what they hold need not be zero), blocks past it, or on a bad page, come from outside the
//    pool, where TMA fills in zeros;
//  - CTAs stay and take the next blocks' jobs (cluster launch control), so ragged lengths even out;
//  - the streams' results are merged from tensor memory, where both of a row lie in the same lane: half of
//    the dims by either stream's warps. With one split that is the result, else it goes to the
//    workspace and paged_join_kernel joins the splits.
#include <string.h>

#include <numeric>

#include "hsa_flash.cuh"
#include "hsa_paged.cuh"

namespace hsa {
namespace {

constexpr int kTile = 128;               // query rows
constexpr int kKeys = 64;                // keys of a tile
constexpr int kSoftWarps = 8;            // 4 per stream: two warp groups; the third holds the other roles
constexpr int kMmaWarp = 8, kLoadWarp = 10;              // a warp per stream's products; warp 11 finds the work
constexpr int kThreads = 12 * 32;
constexpr int kSoftRegs = 208, kOtherRegs = 88;          // as in the prompt kernel: 2 x 208 + 88 = 3 x 168 at launch
constexpr uint32_t kBlockQ = kTile * 128, kBlockK = kKeys * 128;   // 64 dims of a tile, 128 bytes a row
constexpr int kJobSlots = 2;

template <int D>
struct Shape {
  static constexpr uint32_t kQBytes = (D / 64) * kBlockQ, kKvBytes = (D / 64) * kBlockK;
  static constexpr int kStages = D == 128 ? 4 : 8;               // tiles of K and V in a stream's ring
  static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kQBytes;     // Q of two jobs
  static constexpr uint32_t kOffStage = kOffKv + 2 * kStages * kKvBytes, kSmem = kOffStage + kSoftWarps * 2048 + 1024;   // + alignment slack
};

struct RowsParams {
  CUtensorMap qm, km, vm;
  PagedAttnParams a;
  int32_t tt;                            // queries per chunk: 128 / group
  int32_t box;                           // rows of a box of the pools
  uint64_t wait_ns;
};

struct Job {
  int b, h, chunk, split, lo, hi;        // [lo, hi): the positions that queries of the request see
  int j0[2], j1[2];                      // 64-key tiles [j0, j1) of stream t
  int whole;                             // the request's only split
  int more;                              // 0: no work is left, the other fields are not set
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const __grid_constant__ RowsParams rp) {
  using L = Shape<D>;
  const PagedAttnParams& p = rp.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Job s_job[kJobSlots];
  __shared__ float2 s_ml[2][2][kTile];                   // of jobs in turn, each stream's (m in log2 units, l) of a row
  __shared__ __align__(16) uint4 s_answer;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bars[25 + 2 * kJobSlots + 4 * L::kStages];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base + L::kOffQ, sKv = base + L::kOffKv;
  // mbarriers: Q loaded / read by both streams' last products, for jobs in turn; for each stream O read,
  // every product done; two for each stream, for key tiles in turn: S computed, P written, P V added to O.
  // Then the two warps of 32 rows meeting, the launcher's answer, the jobs and the rings
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t q_full = bars, q_empty = bars + 16, o_empty = bars + 32, drain = bars + 48, s_full = bars + 64, p_full = bars + 96,
                 o_full = bars + 128, pair = bars + 160, answered = bars + 192, job_full = bars + 200, job_empty = job_full + 8 * kJobSlots,
                 kv_full = job_empty + 8 * kJobSlots, kv_empty = kv_full + 16 * L::kStages;
  static_assert(200 + 16 * kJobSlots + 32 * L::kStages <= sizeof(s_bars), "barriers");

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + 8 * t, 1);
      mbar_init(q_empty + 8 * t, 2);
      mbar_init(o_empty + 8 * t, kSoftWarps);
      mbar_init(drain + 8 * t, 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full + 16 * t + 8 * b, 1);
        mbar_init(p_full + 16 * t + 8 * b, 4);
        mbar_init(o_full + 16 * t + 8 * b, 1);
      }
    }
    for (int w = 0; w < 4; ++w) mbar_init(pair + 8 * w, 2);
    mbar_init(answered, 1);
    for (int s = 0; s < kJobSlots; ++s) {
      mbar_init(job_full + 8 * s, 1);
      mbar_init(job_empty + 8 * s, kSoftWarps + 3);
    }
    for (int s = 0; s < 2 * L::kStages; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 1);
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
    ok = wait_bar(job_full + 8 * s, (it / kJobSlots) & 1, rp.wait_ns) && ok;
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
      // Lane (block, part) of a tile issues one box: `box` positions x 64 dims. Both streams' rings hold
      // K(0) K(1) V(0) K(2) V(1) ... V(n-1): the products of S run a tile ahead of those with V.
      const int blocks = kKeys / rp.box, part = lane % (D / 64), block = lane / (D / 64);
      int n_q = 0, c[2] = {0, 0};        // queries loaded; tiles of each ring loaded
      Job job;
      // Pages of 32 / blocks tiles at a time, one block per lane, looked up a turn ahead; n_pages: no page
      // (TMA then fills in zeros)
      const int per = 32 / blocks;
      int pages[2], pages_next[2];
      auto find_pages = [&](int t, int turn) {
        const int j = job.j0[t] + turn * per + lane / blocks, pos = kKeys * j + rp.box * (lane % blocks);
        int page = (int)p.n_pages;
        if (j < job.j1[t] && pos < job.hi && pos + rp.box > job.lo) {
          const int x = p.table[(int64_t)job.b * p.max_pages + pos / p.page_size];
          if (x >= 0 && x < p.n_pages)
            page = x;
          else
            flag_status(p.status, HSA_FLAG_INDEX_RANGE);
        }
        return page;
      };
      auto page_of = [&](int t, int i) {   // of this lane's block of tile j0 + i; called with i = 0, 1, 2, ...
        if (i > 0 && i % per == 0) {
          pages[t] = pages_next[t];
          pages_next[t] = find_pages(t, i / per + 1);
        }
        return __shfl_sync(0xffffffffu, pages[t], (i % per) * blocks + block % blocks);
      };
      auto load_kv = [&](int t, int j, int page, const CUtensorMap* map) {
        const int s = c[t] % L::kStages;
        const uint32_t bar = 8 * (t * L::kStages + s);
        ok = ok && wait_bar(kv_empty + bar, ((c[t] / L::kStages) & 1) ^ 1, rp.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(kv_full + bar, L::kKvBytes);
        __syncwarp();
        if (block < blocks)
          tma_4d(sKv + (t * L::kStages + s) * L::kKvBytes + part * kBlockK + (uint32_t)(block * rp.box) * 128u, map, 64 * part,
                 (kKeys * j + rp.box * block) % p.page_size, job.h, page, kv_full + bar);
        ++c[t];
      };
      for (int it = 0; take_job(it, job); ++it) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          pages[t] = find_pages(t, 0);
          pages_next[t] = find_pages(t, 1);
        }
        const int qs = it & 1;
        ok = wait_bar(q_empty + 8 * qs, ((it >> 1) & 1) ^ 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + 8 * qs, (D / 64) * (uint32_t)(rp.tt * p.group) * 128u);
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            tma_4d(sQ + qs * L::kQBytes + d * kBlockQ, &rp.qm, 64 * d, 0, job.h, job.b * p.nq + job.chunk * rp.tt, q_full + 8 * qs);
        }
        ++n_q;
        int at[2] = {0, 0}, ahead[2] = {0, 0};       // pages of the tiles whose V and K come next
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (job.j0[t] < job.j1[t]) {
            at[t] = page_of(t, 0);
            load_kv(t, job.j0[t], at[t], &rp.km);
          }
        const int n = max(job.j1[0] - job.j0[0], job.j1[1] - job.j0[1]);
        for (int i = 0; i < n && ok; ++i) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (job.j0[t] + i + 1 < job.j1[t] && ok) {
              ahead[t] = page_of(t, i + 1);
              load_kv(t, job.j0[t] + i + 1, ahead[t], &rp.km);
            }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (job.j0[t] + i < job.j1[t] && ok) load_kv(t, job.j0[t] + i, at[t], &rp.vm);
            at[t] = ahead[t];
          }
        }
        if (!ok) break;
      }
      // nothing of this CTA's may be in flight when it ends, whatever the other roles did
#pragma unroll
      for (int t = 0; t < 2; ++t)
        for (int e = max(0, c[t] - L::kStages); e < c[t]; ++e)
          ok = drain_bar(kv_full + 8 * (t * L::kStages + e % L::kStages), (e / L::kStages) & 1) && ok;
      for (int e = max(0, n_q - 2); e < n_q; ++e) ok = drain_bar(q_full + 8 * (e & 1), (e >> 1) & 1) && ok;
    } else if (warp < kLoadWarp) {
      // -------------------------------------------------------------- products of one stream
      const int t = warp - kMmaWarp;
      const uint32_t tS = tmem + 128 * t, tO = tmem + 256 + 128 * t, ring = sKv + t * L::kStages * L::kKvBytes;
      const uint32_t full = kv_full + 8 * t * L::kStages, empty = kv_empty + 8 * t * L::kStages;
      const uint32_t id_qk = idesc_f16(kTile, kKeys, false, false, BF16), id_pv = idesc_f16(kTile, D, false, true, BF16);
      const uint32_t one = elect_one();
      auto wait = [&](uint32_t bar, int n) {
        ok = wait_bar(bar, n & 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return ok;
      };
      int n_s = 0, n_p = 0, c = 0;       // key tiles of S and P, tiles of the ring
      auto wait_kv = [&]() { return wait(full + 8 * (c % L::kStages), c / L::kStages); };
      auto free_kv = [&]() {
        umma_commit_one(one, empty + 8 * (c % L::kStages));
        ++c;
      };
      auto qk = [&](int it) {
        const uint64_t dq = sdesc(sQ + (it & 1) * L::kQBytes, 16u, 1024u);
        const uint64_t dk = sdesc(ring + (c % L::kStages) * L::kKvBytes, 16u, 1024u);
        const uint32_t at = tS + 64 * (n_s & 1);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss(one, at, dq + (((k >> 2) * kBlockQ + (k & 3) * 32u) >> 4), dk + (((k >> 2) * kBlockK + (k & 3) * 32u) >> 4), id_qk,
                  k > 0);
        umma_commit_one(one, s_full + 16 * t + 8 * (n_s & 1));
        ++n_s;
      };
      auto pv = [&](bool acc) {
        const uint64_t dv = sdesc(ring + (c % L::kStages) * L::kKvBytes, kBlockK, 1024u);
        const uint32_t at = tS + 64 * (n_p & 1);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) umma_ts(one, tO, at + 8 * k, dv + ((k * 16u * 128u) >> 4), id_pv, acc || k > 0);
        umma_commit_one(one, o_full + 16 * t + 8 * (n_p & 1));
        ++n_p;
      };
      Job job;
      for (int it = 0; take_job(it, job); ++it) {
        const int j0 = uniform(t ? job.j0[1] : job.j0[0]), j1 = uniform(t ? job.j1[1] : job.j1[0]);
        const int lo = uniform(job.lo), hi = uniform(job.hi);
        if (!wait(q_full + 8 * (it & 1), it >> 1)) break;
        if (j0 < j1) {
          if (!wait_kv()) break;
          qk(it);
          free_kv();
        }
        for (int j = j0; j < j1 && ok; ++j) {
          if (j + 1 < j1) {
            if (!wait_kv()) break;
            qk(it);
            free_kv();
          }
          if (j + 1 == j1) umma_commit_one(one, q_empty + 8 * (it & 1));   // Q's last product is issued
          if (!wait_kv()) break;
          const int first = max(0, lo - kKeys * j), end = min(kKeys, hi - kKeys * j);   // rows that some query sees
          if (first > 0 || end < kKeys) {
            const uint32_t v = ring + (c % L::kStages) * L::kKvBytes;
            for (int x = lane; x < kKeys * 8; x += 32)
              if ((x >> 3) < first || (x >> 3) >= end)
#pragma unroll
                for (int d = 0; d < D / 64; ++d) sts128(v + d * kBlockK + x * 16u, 0u, 0u, 0u, 0u);
            fence_async_smem();
            __syncwarp();
          }
          // the first product of a job overwrites O: the last job's must have been read
          if (j == j0 && !wait(o_empty + 8 * t, it ^ 1)) break;
          if (!wait(p_full + 16 * t + 8 * (n_p & 1), n_p >> 1)) break;
          pv(j > j0);
          free_kv();
        }
        if (!ok) break;
        if (j0 == j1) umma_commit_one(one, q_empty + 8 * (it & 1));
      }
      umma_commit_one(one, drain + 8 * t);       // every product is done before the tensor memory is freed
      ok = drain_bar(drain + 8 * t, 0) && ok;
    } else {
      // -------------------------------------------------------------- what comes next
      // A block is taken only when the work before the last has been done by every role, so that no CTA
      // holds back more than one piece of work (taking three ahead left ragged batches uneven).
      const uint32_t answer = smem_u32(&s_answer);
      uint32_t block = blockIdx.x;
      int it = 0;
      auto wait_slot = [&]() {
        ok = wait_bar(job_empty + 8 * (it % kJobSlots), ((it / kJobSlots) & 1) ^ 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      for (int n = 0; ok; ++n) {
        Job job;
        int idx = (int)block;
        job.chunk = idx % p.chunks;
        idx /= p.chunks;
        job.h = idx % p.heads;
        idx /= p.heads;
        job.b = idx % p.batch;
        job.split = idx / p.batch;
        job.more = 1;
        const Span sp = request_span(p, job.b);
        job.lo = sp.lo;
        job.hi = sp.hi;
        if (lane < p.nq && job.split == 0 && job.h == 0) {
          const int raw = p.vis[(int64_t)job.b * p.nq + lane];
          if (raw != clamp_vis(p, raw)) flag_status(p.status, HSA_FLAG_INDEX_RANGE);
        }
        if (job.split < sp.used) {
          const int begin = (sp.base + job.split * sp.len) / kKeys, end = (min(sp.base + (job.split + 1) * sp.len, sp.hi) + kKeys - 1) / kKeys;
          const int half = (max(0, end - begin) + 1) / 2;
          job.j0[0] = begin;
          job.j1[0] = job.j0[1] = begin + half;
          job.j1[1] = max(end, begin + half);
          job.whole = sp.used == 1;
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
  } else {
    // ---------------------------------------------------------------- softmax: one row per thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * t, tO = tS + 256u;
    const float scale = p.scale_log2;
    const int rows = p.nq * p.group;
    int n_s = 0;                         // key tiles so far
    for (int it = 0; wait_job(it); ++it) {
      const Job& job = s_job[it % kJobSlots];
      const int j0 = t ? job.j0[1] : job.j0[0], j1 = t ? job.j1[1] : job.j1[0], b = job.b, job_hi = job.hi;
      const int row = job.chunk * rp.tt * p.group + r;
      const bool real = r < rp.tt * p.group && row < rows;
      const int h = job.h, partner = t ? job.j1[0] - job.j0[0] : job.j1[1] - job.j0[1];   // the other stream's tiles
      const bool whole = job.whole;
      const int64_t slot = ((int64_t)b * p.heads + h) * p.n_splits + job.split;
      const bool warp_real = (warp & 3) * 32 < rp.tt * p.group && job.chunk * rp.tt * p.group + (warp & 3) * 32 < rows;
      int lo = 0, hi = 0;                // this row's keys
      if (real) {
        hi = clamp_vis(p, p.vis[(int64_t)b * p.nq + row / p.group]);
        lo = p.window > 0 ? max(hi - p.window, 0) : 0;
      }
      const int all_lo = __reduce_max_sync(0xffffffffu, real ? lo : 0), all_hi = __reduce_min_sync(0xffffffffu, real ? hi : 0x7fffffff);
      const bool small = p.page_size < kKeys || p.page_size % kKeys;   // a tile may lie on several pages
      float m = -INFINITY, l = 0.f;
      // pages of the tile's 16-row pieces, looked up a tile ahead by lanes 0..3: a bad one masks its keys
      auto good_of = [&](int j) {
        bool good = true;
        const int pos = kKeys * j + 16 * lane;
        if (warp_real && lane < (small ? 4 : 1) && pos < job_hi) {
          const int x = p.table[(int64_t)b * p.max_pages + pos / p.page_size];
          good = x >= 0 && x < p.n_pages;
        }
        return good;
      };
      bool good = j0 < j1 ? good_of(j0) : true;
      for (int j = j0; j < j1; ++j, ++n_s) {
        const uint32_t bad = __ballot_sync(0xffffffffu, !good);
        if (j + 1 < j1) good = good_of(j + 1);
        ok = wait_bar(s_full + 16 * t + 8 * (n_s & 1), (n_s >> 1) & 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (warp_real) {
          const int hr = hi - kKeys * j, lr = lo - kKeys * j;
          softmax_tile<D, BF16>(
              tS + 64 * (n_s & 1), tO, hr > 0 && lr < kKeys, scale, m, l, j > j0,
              [&](uint32_t(&s)[2][32]) {
                if (kKeys * (j + 1) > all_hi || kKeys * j < all_lo || bad) {
                  const uint32_t hidden = small ? bad : (bad ? 15u : 0u);
#pragma unroll
                  for (int c = 0; c < kKeys; ++c)
                    if (c >= hr || c < lr || ((hidden >> (c >> 4)) & 1u)) s[c >> 5][c & 31] = 0xFF800000u;   // -inf
                }
              },
              [&]() {                    // the last tile's P V is in O
                ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, rp.wait_ns) && ok;
                tc_fence_after();
              });
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * (n_s & 1));
      }
      if (!ok) break;
      // -------------------------------------------------------------- both streams' O and (m, l)
      if (j0 < j1) {
        ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, rp.wait_ns) && ok;   // the last P V
        ok = __all_sync(0xffffffffu, ok);
      }
      const float m2 = m == -INFINITY ? m : m * scale;
      s_ml[it & 1][t][r] = make_float2(m2, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(pair + 8 * (warp & 3));
      ok = ok && wait_bar(pair + 8 * (warp & 3), it & 1, rp.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float2 other = s_ml[it & 1][t ^ 1][r];
      const bool mine_any = m2 != -INFINITY || l != 0.f, other_any = other.x != -INFINITY || other.y != 0.f;
      const float M = fmaxf(m2, other.x);
      const float fm = m2 == -INFINITY ? 0.f : ex2_ftz(m2 - M), fo = other.x == -INFINITY ? 0.f : ex2_ftz(other.x - M);
      const float lsum = (mine_any ? fm * l : 0.f) + (other_any ? fo * other.y : 0.f);
      const float gain = !whole ? 1.f : (lsum != 0.f ? p.v_scale / lsum : 0.f);
      const uint32_t tM = tO + (D / 2) * t, tP = tM + (t ? -128 : 128);   // this warp's half of the dims, in either stream's O
      const int row0 = row - lane, row_end = min(rows, (row - r) + rp.tt * p.group);   // this warp's first row, and past the chunk's last
      const uint32_t stage = base + L::kOffStage + (uint32_t)warp * 2048u;
      free_job(it);
      if (warp_real) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t x[32], y[32];
          if (j0 < j1) TMEM_LD32(tM + 32 * c, x);
          if (partner > 0) TMEM_LD32(tP + 32 * c, y);
          tmem_wait_ld();
          tmem_regs_ready(x);
          tmem_regs_ready(y);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = __float_as_uint(((mine_any ? fm * __uint_as_float(x[e]) : 0.f) + (other_any ? fo * __uint_as_float(y[e]) : 0.f)) * gain);
          // 64 bytes of each row at a time go through shared memory, so that four lanes write them together:
          // this lane then holds piece lane % 4 of rows 8 i + lane / 4
          auto flush = [&](auto&& piece, auto&& place) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 v = piece(e);
              sts128(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), v.x, v.y, v.z, v.w);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int sr = 8 * i + (lane >> 2);
              const uint4 v = lds128(stage + sr * 64 + (((lane & 3) ^ ((sr >> 1) & 3)) << 4));
              if (row0 + sr < row_end) *place(row0 + sr) = v;
            }
            __syncwarp();
          };
          const int d = (D / 2) * t + 32 * c;
          if (!whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
              flush([&](int e) { return make_uint4(x[16 * u + 4 * e], x[16 * u + 4 * e + 1], x[16 * u + 4 * e + 2], x[16 * u + 4 * e + 3]); },
                    [&](int rw) { return reinterpret_cast<uint4*>(p.part_o + (slot * rows + rw) * D + d + 16 * u) + (lane & 3); });
          } else {
            flush(
                [&](int e) {
                  auto two = [&](int i) { return pack2<BF16>(__uint_as_float(x[8 * e + 2 * i]), __uint_as_float(x[8 * e + 2 * i + 1])); };
                  return make_uint4(two(0), two(1), two(2), two(3));
                },
                [&](int rw) {
                  const int64_t at = ((int64_t)b * p.nq + rw / p.group) * p.heads_q + h * p.group + rw % p.group;
                  return reinterpret_cast<uint4*>(p.out + at * D + d) + (lane & 3);
                });
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_empty);
        mbar_arrive(o_empty + 8);
      }
      if (real && t == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * rows + row)) = make_float2(M, lsum);
        else if (p.lse)
          p.lse[((int64_t)b * p.nq + row / p.group) * p.heads_q + h * p.group + row % p.group] = lsum != 0.f ? (M + log2f(lsum)) * kLn2 : -INFINITY;
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
cudaError_t launch(const RowsParams& p, unsigned blocks, cudaStream_t s) {
  auto kernel = paged_rows_kernel<D, BF16>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), Shape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), Shape<D>::kSmem, s, p);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedAttnParams& a, int32_t head_dim, int32_t kv_dtype, uint64_t wait_ns, cudaStream_t s) {
  const TensorMapEncoder encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  RowsParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.tt = kTile / a.group;
  p.box = std::gcd(a.page_size, kKeys);
  p.wait_ns = wait_ns;
  const CUtensorMapDataType type = kv_dtype == HSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t d = (cuuint64_t)head_dim;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  {
    // q as [request and query][key-value head][head of the group][dim]: a box is tt queries x the group x 64 dims
    const cuuint64_t dims[4] = {d, (cuuint64_t)a.group, (cuuint64_t)a.heads, (cuuint64_t)a.batch * a.nq};
    const cuuint64_t strides[3] = {2 * d, 2 * d * a.group, 2 * d * a.heads_q};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.group, 1, (cuuint32_t)p.tt};
    if (encode(&p.qm, type, 4, const_cast<uint16_t*>(a.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    // the pools as [page][head][position][dim]: a box is `box` positions x 64 dims
    const cuuint64_t dims[4] = {d, (cuuint64_t)a.page_size, (cuuint64_t)a.heads, (cuuint64_t)a.n_pages};
    const cuuint64_t strides[3] = {2 * d, 2 * d * a.page_size, 2 * d * a.page_size * a.heads};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
    if (encode(i ? &p.vm : &p.km, type, 4, const_cast<uint8_t*>(i ? a.v_pool : a.k_pool), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const unsigned blocks = (unsigned)a.n_splits * a.batch * a.heads * a.chunks;
  if (head_dim == 128) return kv_dtype == HSA_BF16 ? launch<128, true>(p, blocks, s) : launch<128, false>(p, blocks, s);
  return kv_dtype == HSA_BF16 ? launch<64, true>(p, blocks, s) : launch<64, false>(p, blocks, s);
}

}  // namespace hsa
