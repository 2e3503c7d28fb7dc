// Verification of a draft against the target's probabilities (hsa_draft_verify): x_i stays while u_i q_i(x_i) < p_i(x_i); at the
// first that does not, row a, the next token is drawn from w = max(0, p_a - q_a), behind the last from w = p_a: the lowest v
// whose running sum passes u times the sum of w.
//
// Bound: one row of p, and of q, per request is read (of nq each, the others only at one place); for one request it is
// the chain of dependent loads: the draft, its probabilities, the row, the piece of it that holds the token.
//  - A request gets a cluster of up to 8 CTAs. Each finds a by itself (a lane per drafted token), then sums its share of
//    the row, a contiguous piece for each warp; the CTAs exchange their sums through distributed shared memory, and the
//    CTA whose share holds the border finds the warp's piece, which all its threads then go through once more (from L2).
//  - Sums are integers in units of 2^-46, so that neither the cut into pieces nor the order of anything changes a token.
//    (The borders of sums in fp32 would move by more than most tokens weigh; fp64 adds are slower than the
//    loads here.) An entry becomes two integers by four fp32 additions: the bits of 1 + x hold x in units of 2^-23, and
//    the rest, which fp32 holds exactly, gives 23 more bits in the same way.
// Measured, 131,072 entries, fp32: 1 request x 5 rows 6.0 us, 64 requests 15.6 us, 0.55 of the measured copy rate (rows of 131,071, read entry by
// entry: 18), 200 requests 38 us, 0.71; bf16: 100 x 4 rows 17.3 us, 0.39; 37 lookups x 8 rows of 50,001 bf16 entries 5.7 us. What is left in the
// short ones is the launch, the cluster's start and loads that wait for one another; with 16-bit entries also the sums, which take 10
// instructions for each of 2 bytes as they take 11 for each of 4 (issue 50 % of the active clocks against 33, HBM 26 % against 38).
#include <string.h>

#include "hsa_common.cuh"
#include "hsa_dense.h"

namespace hsa {
namespace {

constexpr int kStep = 128;               // pieces are multiples of this many entries
// CTAs of 256 threads that an SM holds. 16-bit entries: batches of 8 and 3 CTAs, of 4 and 4, of 2 and 4: 100 x 4 rows of 131,072 17.6, 21.1, 21.9 us;
// fp32: batches of 4 and 4 CTAs, of 8 and 3: 64 x 5 rows 16.0, 19.0
template <typename T>
constexpr int kCtas = sizeof(T) == 4 ? 4 : 3;
constexpr int kFlush = 128;              // entries of a lane between 64-bit sums, at most: low parts are 2^22 for p and for q

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value_of(__half x) { return __half2float(x); }

// x of [0, 1] to the nearest multiple of 2^-46: hi 2^-23 + lo 2^-46, |lo| <= 2^22. `hi` and `lo` carry the
// bits of kHi and kLo besides, which a difference takes out.
constexpr float kHi = 1.f, kLo = 0x1.8p-23f;
struct Fixed {
  int hi, lo;
};
__device__ __forceinline__ Fixed fixed_of(float x) {
  const float a = __fadd_rn(x, kHi);
  const float rest = __fsub_rn(x, __fsub_rn(a, kHi));    // exact
  return {__float_as_int(a), __float_as_int(__fadd_rn(rest, kLo))};
}
constexpr Fixed kZero = {0x3F800000, 0x34400000};        // fixed_of(0): the bits of kHi and kLo
// Two at a time, by the packed additions (which round like the single ones)
__device__ __forceinline__ void fixed_of2(float x, float y, Fixed& f, Fixed& g) {
  const uint64_t v = f2_pack(x, y), a = f2_add(v, f2_pack(kHi, kHi));
  const uint64_t b = f2_add(f2_fma(f2_add(a, f2_pack(-kHi, -kHi)), f2_pack(-1.f, -1.f), v), f2_pack(kLo, kLo));
  float lo, hi;
  f2_unpack(a, lo, hi);
  f.hi = __float_as_int(lo);
  g.hi = __float_as_int(hi);
  f2_unpack(b, lo, hi);
  f.lo = __float_as_int(lo);
  g.lo = __float_as_int(hi);
}

// What the next token is drawn from: entry v weighs p[v] - q[v] (Q), p[v] but for v = without (else), as far as above 0
template <typename T, bool Q>
struct Weights {
  const T* p;
  const T* q;
  int without;
  __device__ __forceinline__ void add(float x, Fixed f, float y, Fixed g, int v, int& hi, int& lo) const {
    if constexpr (Q) {
      if (x > y) {
        hi += f.hi - g.hi;
        lo += f.lo - g.lo;
      }
    } else if (v != without) {
      hi += f.hi - kZero.hi;
      lo += f.lo - kZero.lo;
    }
  }
  // adds the weight of v, whose entries are a and b, in two parts
  __device__ __forceinline__ void add(T a, T b, int v, int& hi, int& lo) const {
    const float x = __saturatef(value_of(a)), y = Q ? __saturatef(value_of(b)) : 0.f;          // NaN: 0
    add(x, fixed_of(x), y, Q ? fixed_of(y) : kZero, v, hi, lo);
  }
  // the same for v and v + 1
  __device__ __forceinline__ void add2(T a0, T a1, T b0, T b1, int v, int& hi, int& lo) const {
    const float x0 = __saturatef(value_of(a0)), x1 = __saturatef(value_of(a1));
    const float y0 = Q ? __saturatef(value_of(b0)) : 0.f, y1 = Q ? __saturatef(value_of(b1)) : 0.f;
    Fixed f0, f1, g0 = kZero, g1 = kZero;
    fixed_of2(x0, x1, f0, f1);
    if constexpr (Q) fixed_of2(y0, y1, g0, g1);
    add(x0, f0, y0, g0, v, hi, lo);
    add(x1, f1, y1, g1, v + 1, hi, lo);
  }
  __device__ __forceinline__ int64_t at(int v) const {
    int hi = 0, lo = 0;
    add(p[v], Q ? q[v] : p[v], v, hi, lo);
    return ((int64_t)hi << 23) + lo;
  }
};

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Lane l: the sum over lanes 0 .. l
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The sum of the weights of [lo, hi), by a warp. The loads of a batch go before anything that needs them.
template <typename T, bool WIDE, bool Q>
__device__ __forceinline__ int64_t sum_piece(const Weights<T, Q>& w, int lo, int hi, int lane) {
  int64_t sum = 0;
  if constexpr (WIDE) {                  // 16 bytes at a time; lo is a multiple of kStep
    constexpr int kPer = 16 / sizeof(T), kBatch = sizeof(T) == 4 ? 4 : 8;
    static_assert(kPer * kBatch <= kFlush, "low parts");
    const int n = (hi - lo) / kPer;
    const uint4* p = reinterpret_cast<const uint4*>(w.p + lo);
    const uint4* q = reinterpret_cast<const uint4*>(w.q + lo);
    // a batch of which some vectors lie behind the end spares those, which a whole one does not ask for
    auto batch = [&](int first, bool whole) {
      uint4 a[kBatch], b[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = first + 32 * i;
        a[i] = whole || k < n ? p[k] : make_uint4(0u, 0u, 0u, 0u);
        b[i] = Q && (whole || k < n) ? q[k] : make_uint4(0u, 0u, 0u, 0u);
      }
      int h = 0, l = 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (!whole && first - lane + 32 * i >= n) break;
        T x[kPer], y[kPer];
        memcpy(x, &a[i], 16);
        memcpy(y, &b[i], 16);
#pragma unroll
        for (int e = 0; e < kPer; e += 2) w.add2(x[e], x[e + 1], y[e], y[e + 1], lo + (first + 32 * i) * kPer + e, h, l);
      }
      sum += ((int64_t)h << 23) + l;
    };
    int first = lane;
    for (; first - lane + 32 * kBatch <= n; first += 32 * kBatch) batch(first, true);
    if (first - lane < n) batch(first, false);
    lo += n * kPer;
  }
  constexpr int kBatch = 16;
  for (int first = lo + lane; first < hi; first += 32 * kBatch) {
    T x[kBatch], y[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int v = first + 32 * i;
      x[i] = v < hi ? w.p[v] : T(0.f);
      y[i] = Q && v < hi ? w.q[v] : T(0.f);
    }
    int h = 0, l = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w.add(x[i], y[i], first + 32 * i, h, l);
    sum += ((int64_t)h << 23) + l;
  }
  return warp_sum(sum);
}

template <typename T, bool WIDE, int kThreads>
__global__ void __launch_bounds__(kThreads, kCtas<T> * 256 / kThreads) draft_verify_kernel(const __grid_constant__ VerifyParams vp) {
  constexpr int kWarps = kThreads / 32;
  const hsa_verify_args& p = vp.a;
  __shared__ int s_kept, s_without;
  __shared__ int64_t s_piece[kWarps], s_scan[kWarps];    // sums of the warps' pieces; of the warps' parts of one piece
  __shared__ uint64_t s_cta;             // of this CTA's share, which the others read
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ctas = vp.ctas;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas, most = p.nq - 1;
  // everything that depends on nothing is asked for at once
  const int n = p.n_draft ? p.n_draft[b] : most;
  const float u_sample = p.u_sample[b];
  int x = -1;
  float u = 0.f;
  if (warp == 0 && lane < most) {
    x = p.drafted[(int64_t)b * most + lane];
    u = p.u_accept[(int64_t)b * most + lane];
  }
  if (n < 0 || n > most) {               // the same in every CTA of the cluster
    if (n != -1 && rank == 0 && tid == 0) flag_status(vp.status, HSA_FLAG_INDEX_RANGE);
    return;
  }
  const T* rows_p = static_cast<const T*>(p.p) + (int64_t)b * p.nq * p.p_stride;
  const T* rows_q = p.q ? static_cast<const T*>(p.q) + (int64_t)b * most * p.q_stride : nullptr;
  // ---------------------------------------------------------------- how many stay
  if (warp == 0) {
    const bool known = lane >= n || (x >= 0 && x < p.vocabulary);
    bool turned = lane < n;
    if (lane < n && known) {
      const T tp = rows_p[lane * p.p_stride + x], tq = rows_q ? rows_q[lane * p.q_stride + x] : T(1.f);
      turned = !((double)u * (double)__saturatef(value_of(tq)) < (double)__saturatef(value_of(tp)));
    }
    const uint32_t all = __ballot_sync(0xffffffffu, turned);
    const int kept = all ? __ffs(all) - 1 : n;
    const int at = __shfl_sync(0xffffffffu, x, kept);
    if (lane == 0) {
      s_kept = kept;
      s_without = kept < n && !rows_q ? at : -1;         // not a token where x is unknown
    }
    if (rank == 0) {
      if (!known && lane == kept) flag_status(vp.status, HSA_FLAG_INDEX_RANGE);
      if (lane == 0) p.accepted[b] = kept;
      if (lane < p.nq && lane != kept) p.tokens[(int64_t)b * p.nq + lane] = lane < kept ? x : -1;
    }
  }
  __syncthreads();
  const int kept = s_kept;
  const T* row_p = rows_p + kept * p.p_stride;
  const int per = ((p.vocabulary + ctas * kWarps - 1) / (ctas * kWarps) + kStep - 1) / kStep * kStep;
  auto begin_of = [&](int piece) { return min(p.vocabulary, (rank * kWarps + piece) * per); };

  // The sums, of pieces, shares and the row, then the piece and the entry that pass the border; false if the row weighs nothing
  bool waiting = false;                  // the others may still read this CTA's sum
  auto sample = [&](auto w) -> bool {
    const int64_t sum = sum_piece<T, WIDE>(w, begin_of(warp), begin_of(warp + 1), lane);
    if (waiting) cluster_wait();
    __syncthreads();                     // s_piece of an earlier turn has been read
    if (lane == 0) s_piece[warp] = sum;
    __syncthreads();
    uint64_t before = 0, total = 0;      // of the CTAs before this one, of all
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += (uint64_t)s_piece[i];
    if (ctas > 1) {
      if (tid == 0) s_cta = total;
      __syncthreads();
      cluster_sync_all();
      total = 0;
      for (int c = 0; c < ctas; ++c) {
        const uint64_t y = ld_cluster_u64(cluster_map(smem_u32(&s_cta), c));
        if (c < rank) before += y;
        total += y;
      }
      __syncwarp();
      cluster_arrive();
      waiting = true;
    }
    if (!total) return false;
    // border = floor(u total), exact: u = m 2^-shift with shift at least 24, so it is below total, whatever that is
    const uint32_t bits = __float_as_uint(fminf(fmaxf(u_sample, 0.f), 0x1.fffffep-1f));        // NaN: 0
    const int shift = 150 - (int)(bits >> 23);
    const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u;
    const uint64_t high = __umul64hi(total, m), low = total * m;
    const uint64_t border = shift < 64 ? (high << (64 - shift)) | (low >> shift) : shift < 128 ? high >> (shift - 64) : 0ull;
    uint64_t rest = border - before;     // the first entry whose running sum in this CTA's share is above this
    int piece = -1;
    if (border >= before) {
      for (int i = 0; i < kWarps; ++i) {
        if (rest < (uint64_t)s_piece[i]) {
          piece = i;
          break;
        }
        rest -= (uint64_t)s_piece[i];
      }
    }
    if (piece >= 0) {                    // the same in all threads of the CTA
      const int lo = begin_of(piece), hi = begin_of(piece + 1), each = (per + kThreads - 1) / kThreads;
      const int v0 = min(hi, lo + tid * each), v1 = min(hi, v0 + each);
      int64_t own = 0;
#pragma unroll 4
      for (int v = v0; v < v1; ++v) own += w.at(v);
      const int64_t upto = warp_scan(own, lane);
      if (lane == 31) s_scan[warp] = upto;
      __syncthreads();
      int64_t sum = upto - own;
      for (int i = 0; i < warp; ++i) sum += s_scan[i];
      if ((uint64_t)sum <= rest && rest < (uint64_t)(sum + own)) {
        for (int v = v0; v < v1; ++v) {
          sum += w.at(v);
          if (rest < (uint64_t)sum) {
            p.tokens[(int64_t)b * p.nq + kept] = v;
            break;
          }
        }
      }
    }
    return true;
  };
  bool found;
  if (rows_q && kept < n)
    found = sample(Weights<T, true>{row_p, rows_q + kept * p.q_stride, -1});
  else
    found = sample(Weights<T, false>{row_p, nullptr, s_without});
  if (!found && kept < n) found = sample(Weights<T, false>{row_p, nullptr, -1});   // nothing is left of p: p itself
  if (!found && rank == 0 && tid == 0) {
    p.tokens[(int64_t)b * p.nq + kept] = -1;
    flag_status(vp.status, HSA_FLAG_NO_WEIGHT);
  }
  __syncwarp();
  if (waiting) cluster_wait();
}

template <typename T, int THREADS>
cudaError_t launch(const VerifyParams& p, cudaStream_t s) {
  auto kernel = p.wide ? draft_verify_kernel<T, true, THREADS> : draft_verify_kernel<T, false, THREADS>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.batch * p.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T>
cudaError_t launch(const VerifyParams& p, bool few, cudaStream_t s) {
  return few ? launch<T, 512>(p, s) : launch<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_draft_verify(const hsa_verify_args& a, uint32_t* status, cudaStream_t s) {
  VerifyParams p;
  p.a = a;
  p.status = status;
  // A request's CTAs: about as many as run at a time, while a share has more than 16 KB; beyond that while it has 48 KB (fp32,
  // 131,072 entries, 200 requests: 1, 2, 4, 8 CTAs 71, 63, 40, 38 us; bf16 62, 35, 29, 34; 32,000 entries 12.8, 11.8, 14.9, 23.1). Few
  // requests: CTAs of 512 threads (1 and 8 requests of 131,072 fp32 entries 6.0 and 6.5 us, with 256 threads 7.3 and 9.4). With 16-bit
  // entries an SM has room for one of them, and clusters of 8 soon do not all run at a time (16 requests: 10.3 us, 17 with 256 threads 7.1)
  const int size = a.dtype == HSA_F32 ? 4 : 2;
  const bool few = (int64_t)a.batch * 8 <= (size == 4 ? kSms : 64);
  const int64_t bytes = (int64_t)a.vocabulary * size;
  p.ctas = 1;
  while (p.ctas < 8 && ((int64_t)2 * p.ctas * a.batch <= 4 * kSms ? bytes / p.ctas > 16384 : bytes / (2 * p.ctas) >= 49152)) p.ctas *= 2;
  p.wide = ((reinterpret_cast<uintptr_t>(a.p) | reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)(a.p_stride * size) |
             (uintptr_t)(a.q ? a.q_stride * size : 0)) & 15) == 0;
  switch (a.dtype) {
    case HSA_F32: return launch<float>(p, few, s);
    case HSA_BF16: return launch<__nv_bfloat16>(p, few, s);
    default: return launch<__half>(p, few, s);
  }
}

}  // namespace hsa
