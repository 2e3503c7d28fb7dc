// Attention of new tokens over a paged cache for many query rows per key-value head (several queries,
// large groups) and 16-bit or 4-bit pages, on tcgen05; paged_attn.cu and paged_four.cu have the forms for few rows, the first
// also that for E4M3.
//   o = sum_j softmax_j(scale q.k_j) v_j over the positions j a query sees.
//
// Bound: the reads of the pages from HBM, as with few rows, as long as the products keep up. The
// warp MMA does not from about 25 rows on: its 8-column tiles of queries are issued and softmaxed by the same few warps.
// Here up to 128 rows (queries x heads of the group) are one
// tile of a tcgen05 product, and the 32 KB of 64 keys take a stream about 700 clocks, in which an SM's share
// of HBM brings half as much. The split of a CTA's job falls into two halves, one for each stream t:
// a ring of K and V tiles, a warp that loads it, a warp that issues the products, a warp group with a query
// row per thread for the softmax, buffers of S and an accumulator in tensor memory; the two streams fill each
// other's waits. A row without a query (35 rows fill 35 of 128) costs nothing but its lane: warps without any
// skip the softmax, no other request's queries are loaded for it, and it takes no shared memory, which the rings get.
//  - K and V tiles come as boxes of gcd(page size, 64) rows by TMA (128-byte swizzle); rows inside a box that
//    no query sees (past the visible length, or between the windows of queries far apart) are cleared before use, as
//    zero times what they hold need not be zero; blocks without any other row, or on a bad page, come from outside
//    the pool, where TMA fills in zeros;
//  - CTAs stay and take the next blocks' jobs (cluster launch control), so ragged lengths even out;
//  - four warps merge the streams' results from tensor memory, where both of a row lie in the same lane (but see below), while the
//    softmax is at the next job. With one split that is the result, else it goes to the workspace and
//    paged_join_kernel joins the splits.
// Measured: 64 requests x 4 heads x 5 queries, f16, 16,384 keys each 328 us, 0.97 of the measured copy rate; of 1 ..
// 4,097 keys 64 us, 0.67 (the CTAs' last jobs do not end together; all with 4,097: 93 us, 0.86); 1 request x 131,072 55 us.
//
// 4-bit pages (FOUR): eight more warps take the place of the loads by TMA. Each brings its 16 keys of a tile by asynchronous
// copies as they lie in the pool, makes f16 of them (codes times scales, exact) and writes them into the rings' tiles. The reads
// are 9/32 of those from 16-bit pages, so they decide no more. 64 keys of 128 dims take 1,215 clocks of an SM, in which the tensor path
// is busy for 59 %, the converting warps for 70 to 80 % (they wait for a free tile in the rest, timed by the clock), and shared memory for
// 912 by count: 32 KB written and 32 read as converted tiles, 9 written and 9 read as they come, 32 KB of queries for the product with K.
//  - Up to 64 query rows the second stream's queries lie 64 rows lower, so that its rows fall to the warps that the first
//    stream's leave idle (64 x 5 queries x 16,384 keys 306 -> 291 us). The merge then goes through shared memory.
//  - Rings of 2, 3, 4 tiles 311, 293, 291 us; 2, 3, 4, 6 slots for what a converting warp brings 348, 291, 295, 309 (the last two take
//    tiles from the rings); twice the pieces for half the converting warps: 416 against 306. Q in tensor memory would spare its reads, but S of two
//    streams twice and their O take all 512 columns.
// Measured: 64 requests x 4 heads x 5 queries x 7 heads, f16, 16,384 keys each 276 us (16-bit pages: 328), of 1 .. 4,097 keys
// 56.6; 16 x 8 heads x 8 queries x 16 heads, bf16, 8,192 keys 82. 64 dims, 16 x 8 heads, 8,192 keys: 28 and 40 rows 63 us, 128 rows 71, where 128
// dims take 73 with 28 rows. Half the bytes and half the conversion save a seventh: the tensor path is busy for 35 %, issue is at 48, HBM at
// 13, so that what a tile of 64 keys costs whatever its dims (barriers, and S on its way out and back) is likely to decide.
#include <string.h>

#include <numeric>

#include "hsa_flash.cuh"
#include "hsa_four.cuh"
#include "hsa_paged_warp.cuh"

namespace hsa {
namespace {

constexpr int kTile = 128;               // query rows
constexpr int kKeys = 64;                // keys of a tile
constexpr int kSoftWarps = 8;            // 4 per stream: two warp groups; the third holds the other roles
constexpr int kMmaWarp = 8, kLoadWarp = 10;              // a warp per stream's products, and one per stream's loads
constexpr int kOutWarp = 12;             // warps 12..15 merge the streams and write
// The roles of the other warps, and registers per thread: at launch (65,536 over the threads, whole groups of 8), then for the
// softmax groups, whose threads hold a row of 64 logits, for the group of the products, the one that writes, and the rest
template <bool FOUR>
struct Roles {                           // 16-bit pages: warps 10 and 11 load, 16 finds the work, 17..19 only fill its warp group
  static constexpr int kFindWarp = 16, kThreads = 20 * 32, kJobReaders = kSoftWarps + 4 + 4, kFilled = 1;
  static constexpr int kLaunchRegs = 96, kSoftRegs = 136, kIssueRegs = 80, kOutRegs = 80, kLastRegs = 48;
  static_assert(2 * kSoftRegs + kIssueRegs + kOutRegs + kLastRegs <= 5 * kLaunchRegs, "setmaxnreg draws on the launch's registers");
};
template <>
struct Roles<true> {                     // 4-bit pages: warp 10 fills its group, 11 finds the work, 16..23 load and convert, four for each stream
  static constexpr int kFindWarp = 11, kThreads = 24 * 32, kJobReaders = kSoftWarps + 2 + 4 + 8, kFilled = 4;
  // (48 for the converting warps keep their conversions between the stores: 276 us against 283 with 56 and 291 with 64, 64 requests x 5
  // queries x 16,384 keys; with 40 they spill, 307)
  static constexpr int kLaunchRegs = 80, kSoftRegs = 112, kIssueRegs = 40, kOutRegs = 104, kLastRegs = 48;
  static_assert(2 * kSoftRegs + kIssueRegs + kOutRegs + 2 * kLastRegs <= 6 * kLaunchRegs, "setmaxnreg draws on the launch's registers");
};
// A warp group goes on with REGS registers per thread, of the LAUNCH that it was launched with
template <int REGS, int LAUNCH>
__device__ __forceinline__ void take_registers() {
  static_assert(REGS % 8 == 0 && REGS >= 24 && REGS <= 256, "setmaxnreg");
  if constexpr (REGS > LAUNCH)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
constexpr int kConvertWarp = 16;
constexpr uint32_t kSumRow = 80;         // bytes from lane to lane of 16 columns that a writing warp hands over (bank spread)
constexpr uint32_t kBlockK = kKeys * 128;                // 64 dims of a tile of keys, 128 bytes a row
constexpr int kJobSlots = 2;
constexpr int kOrdered = 128;            // batches up to this can be worked off by length

template <int D>
struct Shape {
  static constexpr uint32_t kKvBytes = (D / 64) * kBlockK;
  // tiles of K and V in a stream's ring, at most. 4, 5, 6 at 128 dims: 64 requests x 16,384 keys 332, 327.5, 327 us, of
  // 1 .. 4,097 keys 61.3, 60.7, 61.7, 1 request x 131,072 53.6, 53.9, 55.7
  static constexpr int kMaxStages = D == 128 ? 5 : 10;
  // 4-bit pages: a converting warp's slots of a piece of 16 keys, K and V: codes, then scales
  static constexpr int kRawSlots = 3, kRawBytes = 2 * kPagedGroup * (D / 2 + D / 16);
};

constexpr uint32_t smem_most(bool four) { return 227 * 1024 - (four ? 4608 : 4096); }      // but for what is declared in the kernel

struct RowsParams {
  CUtensorMap qm, km, vm;
  PagedAttnParams a;
  int32_t tt;                            // queries per chunk: as many as a request has, at most 128 / group
  int32_t box;                           // rows of a box of the pools
  int32_t q_rows;                        // rows of a query block in shared memory: tt x group, whole groups of 8
  int32_t stages;                        // of a stream's ring: what the queries leave room for
  int32_t ordered;                       // the longest requests come first
  int32_t shift;                         // 4-bit pages: rows that the second stream's queries lie lower in the products, 64 or 0
  int32_t wide;                          // results start on 32-byte boundaries
  uint64_t wait_ns;
};

struct Job {
  int b, h, chunk, split, lo, hi;        // [lo, hi): where the positions lie that queries of the request see
  int gaps;                              // some of them may be seen by none
  int j0[2], j1[2];                      // 64-key tiles [j0, j1) of stream t
  int whole;                             // the request's only split
  int more;                              // 0: no work is left, the other fields are not set
};

template <int D, bool BF16, bool FOUR>
__global__ void __launch_bounds__(Roles<FOUR>::kThreads, 1) paged_rows_kernel(const __grid_constant__ RowsParams rp) {
  using L = Shape<D>;
  using R = Roles<FOUR>;
  const PagedAttnParams& p = rp.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Job s_job[kJobSlots];
  __shared__ int s_pages[FOUR ? 1 : kJobSlots][2][FOUR ? 1 : 32];   // pages of either stream's first tiles
  __shared__ float s_query[2][FOUR ? kTile : 1];         // 4-bit pages: 2^-shift of each row's queries in f16
  // 4-bit pages: which 16-key pieces of a tile are on bad pages or seen by no query, of each stream's tiles in turn. A tile is written 8 after it
  // is read: the rings and S hold 5 key tiles between the two at most
  __shared__ __align__(4) uint8_t s_bad[2][8][4];
  __shared__ float2 s_ml[2][kTile];                      // each stream's (m in log2 units, l) of a row
  __shared__ __align__(16) uint4 s_answer;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(16) int s_len[kOrdered];          // requests' lengths
  __shared__ uint8_t s_order[kOrdered];                  // requests, the longest first
  __shared__ __align__(8) uint64_t s_bars[23 + 2 * kJobSlots + 4 * L::kMaxStages + 8];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  // Q of two jobs, then the rings. A product reads 128 rows from a query block's start: past its own rows it
  // reads on into what follows, and those rows of S are no one's.
  const uint32_t q_block = (uint32_t)rp.q_rows * 128u, q_bytes = (D / 64) * q_block;
  // (4-bit pages: the rings come first, so that products may start `shift` rows before a block.)
  const int stages = rp.stages;
  const uint32_t rings = 2 * (uint32_t)stages * L::kKvBytes;
  const uint32_t sQ = FOUR ? base + rings : base, sKv = FOUR ? base : base + 2 * q_bytes;
  const uint32_t sRaw = sQ + 2 * q_bytes;                                // 4-bit pages: pieces as they lie in the pools, and
  const uint32_t sSum = sRaw + 8 * L::kRawSlots * L::kRawBytes;          // what one writing warp hands to another
  // mbarriers: Q loaded / read by both streams' last products, for jobs in turn; for each stream O and (m, l)
  // read, every product done; two for each stream, for key tiles in turn: S computed, P written, P V added
  // to O. Then (m, l) written by each stream, the launcher's answer, the jobs and the rings
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t q_full = bars, q_empty = bars + 16, o_empty = bars + 32, drain = bars + 48, s_full = bars + 64, p_full = bars + 96,
                 o_full = bars + 128, ml_full = bars + 160, answered = bars + 176, job_full = bars + 184, job_empty = job_full + 8 * kJobSlots,
                 kv_full = job_empty + 8 * kJobSlots, kv_empty = kv_full + 16 * L::kMaxStages,
                 sum_full = kv_empty + 16 * L::kMaxStages, sum_empty = sum_full + 32;
  static_assert(184 + 16 * kJobSlots + 32 * L::kMaxStages + 64 <= sizeof(s_bars), "barriers");

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + 8 * t, FOUR ? 8 : 1);
      mbar_init(q_empty + 8 * t, 2);
      mbar_init(o_empty + 8 * t, 4);
      mbar_init(ml_full + 8 * t, 4);
      mbar_init(drain + 8 * t, 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full + 16 * t + 8 * b, 1);
        mbar_init(p_full + 16 * t + 8 * b, 4);
        mbar_init(o_full + 16 * t + 8 * b, 1);
      }
    }
    mbar_init(answered, 1);
    for (int s = 0; s < kJobSlots; ++s) {
      mbar_init(job_full + 8 * s, 1);
      mbar_init(job_empty + 8 * s, R::kJobReaders);
    }
    for (int s = 0; s < 2 * L::kMaxStages; ++s) {
      mbar_init(kv_full + 8 * s, R::kFilled);
      mbar_init(kv_empty + 8 * s, 1);
    }
    if constexpr (FOUR)
      for (int s = 0; s < 8; ++s) mbar_init(sum_full + 8 * s, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
  griddep_wait();
  griddep_launch_dependents();
  bool ok = true;
  if (rp.ordered) {                      // four threads for each request count the longer ones
    const int b = tid >> 2;
    if (tid < kOrdered) {
      s_len[tid] = -1;
      if (tid < p.batch) {
        const Span sp = request_span(p, tid);
        s_len[tid] = sp.hi - sp.base;
      }
    }
    __syncthreads();
    if (b < kOrdered) {
      const int mine = s_len[b];
      int before = 0;
      for (int o = 4 * (tid & 3); o < p.batch; o += 16) {
        const int4 x = *reinterpret_cast<const int4*>(s_len + o);
        before += (x.x > mine || (x.x == mine && o < b)) + (x.y > mine || (x.y == mine && o + 1 < b)) +
                  (x.z > mine || (x.z == mine && o + 2 < b)) + (x.w > mine || (x.w == mine && o + 3 < b));
      }
      before += __shfl_xor_sync(0xffffffffu, before, 1);
      before += __shfl_xor_sync(0xffffffffu, before, 2);
      if (b < p.batch && (tid & 3) == 0) s_order[before] = (uint8_t)b;
    }
    __syncthreads();
  }

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

  // Pages of 32 / blocks tiles of a stream at a time, one block per lane, looked up a turn ahead (the first turn's
  // when the job is posted: two reads that depend on each other, which would leave the memory idle between
  // jobs); n_pages: no page (TMA then fills in zeros)
  const int blocks = kKeys / rp.box, per = 32 / blocks;
  auto seen_at = [&](const Job& job, int pos) { return seen32(p, job.b, job.lo, job.hi, job.gaps, pos); };
  auto any_seen = [&](const Job& job, int pos) {         // of a box
    return (seen_at(job, pos) & bits32(0, rp.box)) || (rp.box > 32 && seen_at(job, pos + 32));
  };
  auto find_pages = [&](const Job& job, int j0, int j1, int turn) {
    const int j = j0 + turn * per + lane / blocks, pos = kKeys * j + rp.box * (lane % blocks);
    int page = (int)p.n_pages;
    if (j < j1 && pos < job.hi && pos + rp.box > job.lo && (!job.gaps || any_seen(job, pos))) {
      const int x = p.table[(int64_t)job.b * p.max_pages + pos / p.page_size];
      if (x >= 0 && x < p.n_pages)
        page = x;
      else
        flag_status(p.status, HSA_FLAG_INDEX_RANGE);
    }
    return page;
  };

  // ---------------------------------------------------------------- what comes next
  auto find_work = [&]() {
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
      if (rp.ordered) job.b = s_order[job.b];
      job.split = idx / p.batch;
      job.more = 1;
      const Span sp = request_span(p, job.b);
      job.lo = sp.lo;
      job.hi = sp.hi;
      job.gaps = sp.gaps;
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
        int first[2] = {0, 0};
        if constexpr (!FOUR)
#pragma unroll
          for (int t = 0; t < 2; ++t) first[t] = find_pages(job, job.j0[t], job.j1[t], 0);
        if (!wait_slot()) break;
        if constexpr (!FOUR)
#pragma unroll
          for (int t = 0; t < 2; ++t) s_pages[it % kJobSlots][t][lane] = first[t];
        __syncwarp();
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
  };

  // ---------------------------------------------------------------- 4-bit pages: loads, and codes to f16
  // A warp takes 16 keys of each tile of its stream: pieces of K and V come into its own slots by asynchronous copies, up to
  // kRawSlots ahead, and go from there, converted, into the tiles that the products read. Half a row for each lane, whose bytes
  // are 8 neighbouring dims of every scale's group, in K as in V (the pages' orders): one 16-byte piece of the tile each.
  // Rows no query sees become zeros. The eight warps bring a job's queries, too.
  auto convert = [&]() {
    constexpr int kRow = D / 2, kScaleRow = D / 16, kChunks = kRow / 16, kHalf = kPagedGroup * kRow, kScales = kPagedGroup * kScaleRow;
    constexpr int kCopies = kPagedGroup * kChunks / 32, kSlots = L::kRawSlots;
    const int cw = warp - kConvertWarp, t = cw >> 2, part = cw & 3;
    const uint32_t full = kv_full + 8 * t * L::kMaxStages, empty = kv_empty + 8 * t * L::kMaxStages, ring = sKv + t * stages * L::kKvBytes;
    const uint32_t raw = sRaw + cw * kSlots * L::kRawBytes;
    const int64_t page_pieces = (int64_t)p.heads * (p.page_size / kPagedGroup);
    // 16-byte chunk c of row r of a piece: eight lanes' rows lie apart in the banks
    auto raw_at = [](int r, int c) { return (uint32_t)(r * kRow + (kChunks == 4 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) * 16); };
    const int r0 = lane / kChunks, r = lane & 15, half = lane >> 4;
    // this lane's copies of a piece: 16 bytes of every 32 / kChunks-th row of K and V, and one row's scales, of K or of V
    const uint8_t* const k_src = p.k_pool + lane * 16;
    const uint8_t* const v_src = p.v_pool + lane * 16;
    const uint8_t* const s_src = (lane < 16 ? p.k_s : p.v_s) + r * kScaleRow;
    const uint32_t copy_at = raw_at(r0, lane % kChunks), scale_at = 2 * kHalf + lane * kScaleRow;
    // this lane's chunks of a slot, and where its pieces of a tile go: those of group s to to[s % 4] of its 64 dims
    uint32_t from[D / 64], to[4];
#pragma unroll
    for (int v = 0; v < D / 64; ++v) from[v] = raw_at(r, D / 64 * half + v);
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = (uint32_t)(kPagedGroup * part + r) * 128u + ((2 * e + half) ^ (r & 7)) * 16;
    // ---- the job whose pieces are being loaded: the one that is converted, or already the next
    int b = 0, h = 0, j0 = 0, n_load = 0, loads = 0;     // its tiles, and calls of load() for it
    Span sp = {};
    int64_t pieces = 0;                  // where 32 tiles' pieces lie, one per lane
    int next_page = 0;                   // pages of the 32 after them, read and not yet looked at
    uint32_t load_slot = 0, gone = 0;    // slot that the next piece takes; bit s: the piece in slot s is on a bad page or seen by no query
    auto page_of = [&](int of) {
      const int i = 32 * of + lane, pos = kKeys * (j0 + i) + kPagedGroup * part;
      return i < n_load && pos < sp.hi ? p.table[(int64_t)b * p.max_pages + pos / p.page_size] : -1;
    };
    auto pieces_of = [&](int of, int page) -> int64_t {
      const int i = 32 * of + lane, pos = kKeys * (j0 + i) + kPagedGroup * part;
      return i < n_load ? piece_at(p, sp, b, h, page_pieces, pos, pos / p.page_size, page) : 0;
    };
    // the next tile's piece; every call is one group of copies
    auto load = [&]() {
      if (loads < n_load) {
        const int64_t found = __shfl_sync(0xffffffffu, pieces, loads & 31);
        if ((loads & 31) == 31) {
          pieces = pieces_of((loads >> 5) + 1, next_page);
          next_page = page_of((loads >> 5) + 2);
        }
        const uint32_t seen = (uint32_t)found & 0xFFFFu, at = raw + load_slot * L::kRawBytes;
        const uint64_t piece = (uint32_t)(found >> 16);
        const uint8_t* k = k_src + piece * kHalf;
        const uint8_t* v = v_src + piece * kHalf;
        const uint8_t* sc = s_src + piece * kScales;
        gone = seen ? gone & ~(1u << load_slot) : gone | 1u << load_slot;
        if (seen == 0xFFFFu) {
          page_copy_scales<kScaleRow>(at + scale_at, sc, kScaleRow);
#pragma unroll
          for (int u = 0; u < kCopies; ++u) {
            page_copy16(at + copy_at + u * 512, k + u * 512);
            page_copy16(at + kHalf + copy_at + u * 512, v + u * 512);
          }
        } else {
          const bool some = (seen >> r) & 1u;
          page_copy_scales<kScaleRow>(at + scale_at, some ? sc : p.k_s, some ? (uint32_t)kScaleRow : 0u);
#pragma unroll
          for (int u = 0; u < kCopies; ++u) {
            const uint32_t m = (seen >> (r0 + 8 * u)) & 1u ? 16u : 0u;
            page_copy16z(at + copy_at + u * 512, m ? k + u * 512 : p.k_pool, m);
            page_copy16z(at + kHalf + copy_at + u * 512, m ? v + u * 512 : p.v_pool, m);
          }
        }
        load_slot = load_slot + 1 == kSlots ? 0 : load_slot + 1;
      }
      ++loads;
      page_copies_commit();
    };
    // job `it` from here on: its pieces, its queries (16 or 8 lanes to a row, rows in turn over the eight warps)
    auto open = [&](int it) {
      const Job& job = s_job[it % kJobSlots];
      const int chunk = job.chunk, first = chunk * rp.tt * p.group;
      b = job.b;
      h = job.h;
      j0 = t ? job.j0[1] : job.j0[0];
      n_load = (t ? job.j1[1] : job.j1[0]) - j0;
      sp.lo = job.lo;
      sp.hi = job.hi;
      sp.gaps = job.gaps;
      free_job(it);
      loads = 0;
      // what reads global memory goes first: pages, queries of kBatch turns, the first piece
      const int page = page_of(0);
      next_page = page_of(1);
      constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes, kBatch = 2, kStep = 8 * kRowsAt;
      const int qs = it & 1, rows = p.nq * p.group, c = lane % kLanes;
      uint4 x[kBatch];
      auto fetch = [&](int base_row) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = base_row + i * kStep + lane / kLanes, at = first + row;
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row < rp.tt * p.group && at < rows)
            x[i] = *reinterpret_cast<const uint4*>(p.q + (((int64_t)b * p.nq + at / p.group) * p.heads_q + h * p.group + at % p.group) * D + 8 * c);
        }
      };
      int base_row = cw * kRowsAt;
      fetch(base_row);
      pieces = pieces_of(0, page);
      load();
      ok = wait_bar(q_empty + 8 * qs, ((it >> 1) & 1) ^ 1, rp.wait_ns) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      while (base_row < rp.q_rows) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = base_row + i * kStep + lane / kLanes;
          if (base_row + i * kStep >= rp.q_rows) break;
          float shift = 1.f;
          if (p.q_bf16) {
            uint2 y[2] = {make_uint2(x[i].x, x[i].y), make_uint2(x[i].z, x[i].w)};
            queries_to_f16<2, kLanes>(y, shift);
            x[i] = make_uint4(y[0].x, y[0].y, y[1].x, y[1].y);
          }
          if (row < rp.q_rows) {
            sts128(sQ + qs * q_bytes + (c >> 3) * q_block + row * 128 + ((c & 7) ^ (row & 7)) * 16, x[i].x, x[i].y, x[i].z, x[i].w);
            if (c == 0) s_query[qs][row] = shift;
          }
        }
        base_row += kBatch * kStep;
        if (base_row < rp.q_rows) fetch(base_row);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + 8 * qs);
    };

    // ---- tiles, in the order of the products: K(0) K(1) V(0) K(2) V(1) .. V(n - 1)
    int place = 0, round = 0, tiles = 0; // of the ring; key tiles so far
    auto convert_tile = [&](uint32_t at, bool keys) {    // the slot at `at` to the next place of the ring
      uint32_t w[D / 16];                // this lane's codes
#pragma unroll
      for (int v = 0; v < D / 64; ++v) {
        const uint4 x = lds128(at + (keys ? 0 : kHalf) + from[v]);
        w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
      }
      uint32_t c[D / 64];                // the row's scales
      const uint32_t c_at = at + 2 * kHalf + (keys ? 0 : kScales) + r * kScaleRow;
      if constexpr (D == 128) {
        const uint2 x = lds64(c_at);
        c[0] = x.x, c[D / 64 - 1] = x.y;
      } else {
        c[0] = lds32(c_at);
      }
      ok = wait_bar(empty + 8 * place, (round & 1) ^ 1, rp.wait_ns) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const uint32_t dst = ring + place * L::kKvBytes;
      auto store = [&](int s, uint32_t f, int hi, uint32_t y0, uint32_t y1, uint32_t y2, uint32_t y3) {        // the 8 dims of group s
        sts128(dst + to[s & 3] + (s >> 2) * kBlockK, mul_half(f, hi, y0), mul_half(f, hi, y1), mul_half(f, hi, y2), mul_half(f, hi, y3));
      };
      if (keys) {
        // words j and D / 32 + j: dims 0 .. 3 and 4 .. 7 of the lane's eight, of groups 2 j and 2 j + 1
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16x2x4(w[j], x[0], x[1], x[2], x[3]);
          e2m1x8_to_f16x2x4(w[D / 32 + j], y[0], y[1], y[2], y[3]);
          const uint32_t f = e4m3x2_to_f16x2((uint16_t)(c[j >> 1] >> (16 * (j & 1))));
          store(2 * j, f, 0, x[0], x[1], y[0], y[1]);
          store(2 * j + 1, f, 1, x[2], x[3], y[2], y[3]);
        }
      } else {
        // word D / 64 q + j: dims 2 q, 2 q + 1 of the lane's eight, of groups 4 j .. 4 j + 3
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t x[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) e2m1x8_to_f16x2x4(w[D / 64 * q + j], x[q][0], x[q][1], x[q][2], x[q][3]);
          const uint32_t f0 = e4m3x2_to_f16x2((uint16_t)(c[j] & 0xFFFFu)), f1 = e4m3x2_to_f16x2((uint16_t)(c[j] >> 16));
#pragma unroll
          for (int e = 0; e < 4; ++e) store(4 * j + e, e < 2 ? f0 : f1, e & 1, x[0][e], x[1][e], x[2][e], x[3][e]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * place);
      if (++place == stages) {
        place = 0;
        ++round;
      }
    };
    uint32_t slot = 0;                   // of the tile to be converted
    bool opened = false;
    for (int it = 0; opened || wait_job(it); ++it) {
      if (!opened) open(it);
      if (!ok) break;
      while (loads < kSlots) load();
      opened = false;
      const int n = n_load;
      for (int i = 0; i <= n; ++i) {     // K(i), then V(i - 1)
        const uint32_t last = slot == 0 ? kSlots - 1 : slot - 1;
        if (i < n) {
          page_copies_wait<kSlots - 2>();
          __syncwarp();
          if (lane == 0) s_bad[t][tiles & 7][part] = (gone >> slot) & 1u;
          ++tiles;
          convert_tile(raw + slot * L::kRawBytes, true);
        }
        if (i > 0 && ok) {
          convert_tile(raw + last * L::kRawBytes, false);
          // Into the slot of V(i - 1), which every lane has read. Behind this job's last tile come the next job's, if it is there:
          // its pieces and queries are then on their way while the products are at this one
          if (ok && !opened && loads >= n && __all_sync(0xffffffffu, mbar_test(job_full + 8 * ((it + 1) % kJobSlots), ((it + 1) / kJobSlots) & 1)) &&
              s_job[(it + 1) % kJobSlots].more) {
            open(it + 1);
            opened = true;
          } else if (ok) {
            load();
          }
        }
        if (!ok) break;
        slot = i < n ? (slot + 1 == kSlots ? 0 : slot + 1) : slot;
      }
      if (!ok) break;
    }
    page_copies_wait<0>();
  };

  if (warp >= kSoftWarps && warp < kOutWarp) {
    take_registers<R::kIssueRegs, R::kLaunchRegs>();
    if (FOUR && warp >= kLoadWarp) {
      if (warp == R::kFindWarp) find_work();
    } else if (warp >= kLoadWarp) {
      // -------------------------------------------------------------- loads of one stream, the first's with the queries
      // The ring holds K(0) K(1) V(0) K(2) V(1) ... V(n-1): the products of S run a tile ahead of those with V.
      // Issuing the boxes of a 16 KB tile takes a warp 450 ns, longer than the tile's share of HBM: hence a warp per
      // stream, and warp-uniform operands (a lane for each box: 600).
      const int t = warp - kLoadWarp;
      const uint32_t full = kv_full + 8 * t * L::kMaxStages, empty = kv_empty + 8 * t * L::kMaxStages, ring = sKv + t * stages * L::kKvBytes;
      int n_q = 0, c = 0, place = 0, round = 0;      // queries loaded; tiles of the ring loaded, and its place
      Job job;
      int job_h = 0, j0 = 0, j1 = 0;     // the key head, and this stream's tiles
      int2 pages, pages_next;            // (page, row in it) of this lane's block of a turn
      const uint32_t one = elect_one();
      auto rows_of = [&](int turn, int page) {
        return make_int2(page, (kKeys * (j0 + turn * per + lane / blocks) + rp.box * (lane % blocks)) % p.page_size);
      };
      auto page_of = [&](int i) {        // tile j0 + i, block `lane` of it; called with i = 0, 1, 2, ...
        if (i > 0 && (i & (per - 1)) == 0) {
          pages = pages_next;
          pages_next = rows_of(i / per + 1, find_pages(job, j0, j1, i / per + 1));
        }
        const int src = (i & (per - 1)) * blocks + (lane & (blocks - 1));
        return make_int2(__shfl_sync(0xffffffffu, pages.x, src), __shfl_sync(0xffffffffu, pages.y, src));
      };
      auto load_kv = [&](int2 at, const CUtensorMap* map) {
        ok = wait_bar(empty + 8 * place, (round & 1) ^ 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        const uint32_t bar = full + 8 * place, dst = ring + place * L::kKvBytes;
        if (one) mbar_arrive_expect_tx(bar, L::kKvBytes);
        __syncwarp();
        for (int b = 0; b < blocks; ++b) {
          const int page = __shfl_sync(0xffffffffu, at.x, b), row = __shfl_sync(0xffffffffu, at.y, b);
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            tma_4d_one(one, dst + d * kBlockK + (uint32_t)(b * rp.box) * 128u, map, 64 * d, row, job_h, page, bar);
        }
        ++c;
        if (++place == stages) {
          place = 0;
          ++round;
        }
      };
      for (int it = 0; wait_job(it); ++it) {
        job = s_job[it % kJobSlots];
        job_h = uniform(job.h);
        j0 = t ? job.j0[1] : job.j0[0];
        j1 = t ? job.j1[1] : job.j1[0];
        pages = rows_of(0, s_pages[it % kJobSlots][t][lane]);
        free_job(it);
        if (t == 0) {
          const int qs = it & 1;
          ok = wait_bar(q_empty + 8 * qs, ((it >> 1) & 1) ^ 1, rp.wait_ns) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (one) mbar_arrive_expect_tx(q_full + 8 * qs, (D / 64) * (uint32_t)(rp.tt * p.group) * 128u);
          __syncwarp();
          const int q_at = uniform(job.b * p.nq + job.chunk * rp.tt);
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            tma_4d_one(one, sQ + qs * q_bytes + d * q_block, &rp.qm, 64 * d, 0, job_h, q_at, q_full + 8 * qs);
          ++n_q;
        }
        const int n = j1 - j0;
        int2 at = {}, ahead = {};        // pages of the tiles whose V and K come next
        if (n > 0) {
          at = page_of(0);
          load_kv(at, &rp.km);
          pages_next = rows_of(1, find_pages(job, j0, j1, 1));
        }
        for (int i = 0; i < n && ok; ++i) {
          if (i + 1 < n) {
            ahead = page_of(i + 1);
            load_kv(ahead, &rp.km);
          }
          if (ok) load_kv(at, &rp.vm);
          at = ahead;
        }
        if (!ok) break;
      }
      // nothing of this CTA's may be in flight when it ends, whatever the other roles did
      for (int e = max(0, c - stages); e < c; ++e) ok = drain_bar(full + 8 * (e % stages), (e / stages) & 1) && ok;
      for (int e = max(0, n_q - 2); e < n_q; ++e) ok = drain_bar(q_full + 8 * (e & 1), (e >> 1) & 1) && ok;
    } else {
      // -------------------------------------------------------------- products of one stream
      const int t = warp - kMmaWarp;
      const uint32_t tS = tmem + 128 * t, tO = tmem + 256 + 128 * t, ring = sKv + t * stages * L::kKvBytes;
      const uint32_t full = kv_full + 8 * t * L::kMaxStages, empty = kv_empty + 8 * t * L::kMaxStages;
      const uint32_t id_qk = idesc_f16(kTile, kKeys, false, false, BF16), id_pv = idesc_f16(kTile, D, false, true, BF16);
      const uint32_t one = elect_one();
      auto wait = [&](uint32_t bar, int n) {
        ok = wait_bar(bar, n & 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return ok;
      };
      int n_s = 0, n_p = 0, c = 0, turn = 0;     // key tiles of S and P; place in the ring
      auto wait_kv = [&]() { return wait(full + 8 * c, turn); };
      auto free_kv = [&]() {
        umma_commit_one(one, empty + 8 * c);
        if (++c == stages) {
          c = 0;
          ++turn;
        }
      };
      auto qk = [&](int it) {
        const uint64_t dq = sdesc(sQ + (it & 1) * q_bytes - (FOUR && t ? rp.shift * 128u : 0u), 16u, 1024u);
        const uint64_t dk = sdesc(ring + c * L::kKvBytes, 16u, 1024u);
        const uint32_t at = tS + 64 * (n_s & 1);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss(one, at, dq + (((k >> 2) * q_block + (k & 3) * 32u) >> 4), dk + (((k >> 2) * kBlockK + (k & 3) * 32u) >> 4), id_qk,
                  k > 0);
        umma_commit_one(one, s_full + 16 * t + 8 * (n_s & 1));
        ++n_s;
      };
      auto pv = [&](bool acc) {
        const uint64_t dv = sdesc(ring + c * L::kKvBytes, kBlockK, 1024u);
        const uint32_t at = tS + 64 * (n_p & 1);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) umma_ts(one, tO, at + 8 * k, dv + ((k * 16u * 128u) >> 4), id_pv, acc || k > 0);
        umma_commit_one(one, o_full + 16 * t + 8 * (n_p & 1));
        ++n_p;
      };
      Job job;
      for (int it = 0; take_job(it, job); ++it) {
        const int j0 = uniform(t ? job.j0[1] : job.j0[0]), j1 = uniform(t ? job.j1[1] : job.j1[0]);
        const int lo = uniform(job.lo), hi = uniform(job.hi), gaps = uniform(job.gaps);
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
          if (!FOUR && (kKeys * j < lo || kKeys * (j + 1) > hi || gaps)) {   // there may be rows that no query sees
            const uint32_t seen0 = seen_at(job, kKeys * j), seen1 = seen_at(job, kKeys * j + 32);
            const uint32_t v = ring + c * L::kKvBytes;
            for (int x = lane; x < kKeys * 8; x += 32)
              if (!(((x & 256 ? seen1 : seen0) >> ((x >> 3) & 31)) & 1u))
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
    }
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax: one row per thread
    take_registers<R::kSoftRegs, R::kLaunchRegs>();
    const int t = warp >> 2, r0 = (warp & 3) * 32 - (FOUR && t ? rp.shift : 0), r = r0 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * t, tO = tS + 256u;
    float scale = p.scale_log2;
    const int rows = p.nq * p.group;
    int n_s = 0;                         // key tiles so far
    for (int it = 0; wait_job(it); ++it) {
      const Job& job = s_job[it % kJobSlots];
      const int j0 = t ? job.j0[1] : job.j0[0], j1 = t ? job.j1[1] : job.j1[0], b = job.b, job_hi = job.hi;
      const int row = job.chunk * rp.tt * p.group + r;
      const bool real = r >= 0 && r < rp.tt * p.group && row < rows;
      const bool warp_real = r0 >= 0 && r0 < rp.tt * p.group && job.chunk * rp.tt * p.group + r0 < rows;
      int lo = 0, hi = 0;                // this row's keys
      if (real) {
        hi = clamp_vis(p, p.vis[(int64_t)b * p.nq + row / p.group]);
        lo = p.window > 0 ? max(hi - p.window, 0) : 0;
      }
      const int all_lo = __reduce_max_sync(0xffffffffu, real ? lo : 0), all_hi = __reduce_min_sync(0xffffffffu, real ? hi : 0x7fffffff);
      if constexpr (FOUR) {              // before the job is freed: job it + 2 then waits with its queries
        ok = wait_bar(q_full + 8 * (it & 1), (it >> 1) & 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        scale = r >= 0 && r < rp.q_rows ? p.scale_log2 * s_query[it & 1][r] : p.scale_log2;
      }
      free_job(it);
      const bool small = p.page_size < kKeys || p.page_size % kKeys;   // a tile may lie on several pages
      float m = -INFINITY, l = 0.f;
      // pages of the tile's 16-row pieces, looked up a tile ahead by lanes 0..3: a bad one masks its keys. Only the id is
      // read ahead: compared where it is read, it would hold up the tile for as long as the table takes to answer
      auto page_of = [&](int j) {
        int page = 0;
        const int pos = kKeys * j + 16 * lane;
        if (warp_real && lane < (small ? 4 : 1) && pos < job_hi) page = p.table[(int64_t)b * p.max_pages + pos / p.page_size];
        return page;
      };
      int page = !FOUR && j0 < j1 ? page_of(j0) : 0;
      for (int j = j0; j < j1; ++j, ++n_s) {
        uint32_t bad = 0;
        if constexpr (!FOUR) {
          bad = __ballot_sync(0xffffffffu, page < 0 || page >= p.n_pages);
          if (j + 1 < j1) page = page_of(j + 1);
        }
        ok = wait_bar(s_full + 16 * t + 8 * (n_s & 1), (n_s >> 1) & 1, rp.wait_ns) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if constexpr (FOUR) {
          bad = *reinterpret_cast<const volatile uint32_t*>(s_bad[t][n_s & 7]);
          if (bad) bad = (bad & 1) | (bad >> 7 & 2) | (bad >> 14 & 4) | (bad >> 21 & 8);
        }
        if (warp_real) {
          const int hr = hi - kKeys * j, lr = lo - kKeys * j;
          softmax_tile<D, BF16>(
              tS + 64 * (n_s & 1), tO, hr > 0 && lr < kKeys, scale, m, l, j > j0,
              [&](uint32_t(&s)[2][32]) {
                if (kKeys * (j + 1) > all_hi || kKeys * j < all_lo || bad) {
                  const uint32_t hidden = FOUR || small ? bad : (bad ? 15u : 0u);
#pragma unroll
                  for (int c = 0; c < kKeys; ++c)
                    if (c >= hr || c < lr || ((hidden >> (c >> 4)) & 1u)) s[c >> 5][c & 31] = 0xFF800000u;   // -inf
                }
              },
              [&]() {                    // the last tile's P V is in O
                ok = wait_bar(o_full + 16 * t + 8 * ((n_s - 1) & 1), ((n_s - 1) >> 1) & 1, rp.wait_ns) && ok;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
              });
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * (n_s & 1));
      }
      if (!ok) break;
      // (m, l) to the warps that write, when they have read the last job's
      ok = wait_bar(o_empty + 8 * t, (it & 1) ^ 1, rp.wait_ns) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (!FOUR || r >= 0) s_ml[t][r] = make_float2(m == -INFINITY ? m : fmaf(m, scale, -kLift<BF16>), l);
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_full + 8 * t);
    }
  } else if (warp < kOutWarp + 4) {
    // ---------------------------------------------------------------- both streams' O and (m, l), while the softmax is at the next job
    take_registers<R::kOutRegs, R::kLaunchRegs>();
    // `apart`: the second stream's rows are 64 lower, so in the lanes of warps 2 and 3, which hand their part to warps 0 and 1
    const bool apart = FOUR && rp.shift, hands = apart && (warp & 2);
    const int r = (warp & 3) * 32 + lane - (hands ? 64 : 0), rows = p.nq * p.group;
    const uint32_t tO = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u;
    int n_s[2] = {0, 0}, n_c = 0;        // key tiles of either stream so far; pieces handed over
    for (int it = 0; wait_job(it); ++it) {
      const Job& job = s_job[it % kJobSlots];
      const int tiles[2] = {job.j1[0] - job.j0[0], job.j1[1] - job.j0[1]};
      const int row = job.chunk * rp.tt * p.group + r;
      const bool real = r < rp.tt * p.group && row < rows, warp_real = __any_sync(0xffffffffu, real), whole = job.whole;
      const int64_t slot = ((int64_t)job.b * p.heads + job.h) * p.n_splits + job.split;
      const int64_t at = ((int64_t)job.b * p.nq + row / p.group) * p.heads_q + job.h * p.group + row % p.group;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        ok = ok && wait_bar(ml_full + 8 * t, it & 1, rp.wait_ns);
        n_s[t] += tiles[t];
        if (tiles[t] > 0) ok = ok && wait_bar(o_full + 16 * t + 8 * ((n_s[t] - 1) & 1), ((n_s[t] - 1) >> 1) & 1, rp.wait_ns);   // the last P V
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float2 a = s_ml[0][r], b = s_ml[1][r];
      const bool any_a = a.x != -INFINITY || a.y != 0.f, any_b = b.x != -INFINITY || b.y != 0.f;
      const float M = fmaxf(a.x, b.x);
      const float fa = a.x == -INFINITY ? 0.f : ex2_ftz(a.x - M), fb = b.x == -INFINITY ? 0.f : ex2_ftz(b.x - M);
      const float lsum = (any_a ? fa * a.y : 0.f) + (any_b ? fb * b.y : 0.f);
      const float gain = !whole ? 1.f : (lsum != 0.f ? p.v_scale / lsum : 0.f);
      auto done = [&]() {                // O and (m, l) are in registers
        tc_fence_before();
        free_job(it);
        if (lane == 0) {
          mbar_arrive(o_empty);
          mbar_arrive(o_empty + 8);
        }
      };
      if (!warp_real) {
        done();
        continue;
      }
      auto write = [&](int c, uint32_t (&x)[16]) {       // columns 16 c .. of this row
        // each lane writes its own row, 32 bytes at a time where the rows allow it
        if (whole)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = BF16 || (FOUR && p.q_bf16) ? pack2<true>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]))
                                              : pack2<false>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        if (real) {
          uint32_t* dst = whole ? reinterpret_cast<uint32_t*>(p.out + at * D + 16 * c) : reinterpret_cast<uint32_t*>(p.part_o + (slot * rows + row) * D + 16 * c);
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            if (e == 0 || !whole) {
              if (rp.wide) {
                st_global_256(dst + e, x + e);
              } else {
                *reinterpret_cast<uint4*>(dst + e) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                *reinterpret_cast<uint4*>(dst + e + 4) = make_uint4(x[e + 4], x[e + 5], x[e + 6], x[e + 7]);
              }
            }
        }
      };
      if (apart) {
        const bool any = hands ? any_b : any_a;
        const float f = hands ? fb : fa;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c, ++n_c) {
          uint32_t x[16];
          if (tiles[hands ? 1 : 0] > 0) TMEM_LD16(tO + (hands ? 128 : 0) + 16 * c, x);
          tmem_wait_ld();
          tmem_regs_ready(x);
          if (c == D / 16 - 1) done();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = any ? __float_as_uint(f * __uint_as_float(x[e])) : 0u;
          const int turn = 2 * (warp & 1) + (n_c & 1);   // pair of warps, and its buffers in turn
          const uint32_t mine = sSum + (uint32_t)(32 * turn + lane) * kSumRow;
          ok = (hands ? wait_bar(sum_empty + 8 * turn, ((n_c >> 1) & 1) ^ 1, rp.wait_ns) : wait_bar(sum_full + 8 * turn, (n_c >> 1) & 1, rp.wait_ns)) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (hands) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) sts128(mine + 4 * e, x[e], x[e + 1], x[e + 2], x[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const uint4 y = lds128(mine + 4 * e);
              const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) x[e + k] = __float_as_uint((__uint_as_float(x[e + k]) + __uint_as_float(w[k])) * gain);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive((hands ? sum_full : sum_empty) + 8 * turn);
          if (!hands) write(c, x);
        }
        if (!ok) break;
        if (hands) continue;
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t x[16], y[16];
          if (tiles[0] > 0) TMEM_LD16(tO + 16 * c, x);
          if (tiles[1] > 0) TMEM_LD16(tO + 128 + 16 * c, y);
          tmem_wait_ld();
          tmem_regs_ready(x);
          tmem_regs_ready(y);
          if (c == D / 16 - 1) done();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = __float_as_uint(((any_a ? fa * __uint_as_float(x[e]) : 0.f) + (any_b ? fb * __uint_as_float(y[e]) : 0.f)) * gain);
          write(c, x);
        }
      }
      if (real) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * rows + row)) = make_float2(M, lsum);
        else if (p.lse)
          p.lse[at] = lsum != 0.f ? (M + log2f(lsum)) * kLn2 : -INFINITY;
      }
    }
  } else {
    take_registers<R::kLastRegs, R::kLaunchRegs>();
    if constexpr (FOUR)
      convert();
    else if (warp == R::kFindWarp)
      find_work();
  }
  if (!ok) flag_status(p.status, HSA_FLAG_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int D, bool BF16, bool FOUR = false>
cudaError_t launch(RowsParams& p, unsigned blocks, cudaStream_t s) {
  auto kernel = paged_rows_kernel<D, BF16, FOUR>;
  static const bool fits = launches_with(kernel, Roles<FOUR>::kLaunchRegs);
  if (!fits) return cudaErrorInvalidConfiguration;
  p.q_rows = (p.tt * p.a.group + 7) / 8 * 8;
  // Up to 64 rows lie in two warps' lanes. The second stream's lie 64 lower, in the others', whose schedulers have no softmax else
  p.shift = FOUR && p.q_rows <= 64 ? 64 : 0;
  const uint32_t raw = FOUR ? 8 * Shape<D>::kRawSlots * Shape<D>::kRawBytes + (p.shift ? 4 * 32 * kSumRow : 0) : 0;
  const uint32_t room = smem_most(FOUR) - 1024 - raw - 2 * (D / 64) * (uint32_t)p.q_rows * 128u;
  p.stages = (int32_t)(room / (2 * Shape<D>::kKvBytes));
  if (p.stages > Shape<D>::kMaxStages) p.stages = Shape<D>::kMaxStages;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem_most(FOUR));
  if (e != cudaSuccess) return e;
  const uint32_t smem = 1024 + 2 * (D / 64) * (uint32_t)p.q_rows * 128u + 2 * (uint32_t)p.stages * Shape<D>::kKvBytes + raw;   // 1024: to align
  return launch_pdl(kernel, dim3(blocks), dim3(Roles<FOUR>::kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedAttnParams& a, int32_t head_dim, int32_t kv_dtype, uint64_t wait_ns, cudaStream_t s) {
  RowsParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.tt = a.chunk_rows / a.group;
  p.box = std::gcd(a.page_size, kKeys);
  // Whole requests, more of them than SMs: the longest first, so that the last ones to be taken are short (64 requests
  // x 4 heads of 1 .. 4,097 keys 64 us, 72 in the order of the requests; 100 x 4 of up to 1,024 35 and 40; all with
  // 4,097 95.7 and 95.2). Of requests in several splits the first are alike and few gain (within 3 % either way).
  p.ordered = a.batch <= kOrdered && a.n_splits == 1 && (int64_t)a.batch * a.heads * a.chunks > kSms;
  p.wide = ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.part_o)) & 31) == 0;
  p.wait_ns = wait_ns;
  const unsigned blocks = (unsigned)a.n_splits * a.batch * a.heads * a.chunks;
  if (kv_dtype == HSA_E2M1)              // queries and pages are loaded without tensor maps
    return head_dim == 128 ? launch<128, false, true>(p, blocks, s) : launch<64, false, true>(p, blocks, s);
  const TensorMapEncoder encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
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
  if (head_dim == 128) return kv_dtype == HSA_BF16 ? launch<128, true>(p, blocks, s) : launch<128, false>(p, blocks, s);
  return kv_dtype == HSA_BF16 ? launch<64, true>(p, blocks, s) : launch<64, false>(p, blocks, s);
}

}  // namespace hsa
