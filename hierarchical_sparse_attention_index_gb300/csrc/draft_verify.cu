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
#include <string.h>

#include "hsa_common.cuh"
#include "hsa_dense.h"

namespace hsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 128;               // pieces are multiples of this many entries
constexpr int kFlush = 128;              // entries of a lane between 64-bit sums: 128 low parts, of at most 2^22 for p and for q

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

// What the next token is drawn from: entry v weighs p[v] - q[v] (q given), p[v] but for v = without, as far as above 0
template <typename T>
struct Weights {
  const T* p;
  const T* q;
  int without;
  // adds the weight of v, whose entries are a and b, in two parts
  __device__ __forceinline__ void add(T a, T b, int v, int& hi, int& lo) const {
    const float x = __saturatef(value_of(a));            // NaN: 0
    const Fixed f = fixed_of(x);
    if (q) {
      const float y = __saturatef(value_of(b));
      const Fixed g = fixed_of(y);
      if (x > y) {
        hi += f.hi - g.hi;
        lo += f.lo - g.lo;
      }
    } else if (v != without) {
      hi += f.hi - kZero.hi;
      lo += f.lo - kZero.lo;
    }
  }
  __device__ __forceinline__ int64_t at(int v) const {
    int hi = 0, lo = 0;
    add(p[v], q ? q[v] : p[v], v, hi, lo);
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

// The sum of the weights of [lo, hi), by a warp
template <typename T, bool WIDE>
__device__ __forceinline__ int64_t sum_piece(const Weights<T>& w, int lo, int hi, int lane) {
  int64_t sum = 0;
  if constexpr (WIDE) {                  // 16 bytes at a time; lo is a multiple of kStep
    constexpr int kPer = 16 / sizeof(T), kTurn = kFlush / kPer;
    const int n = (hi - lo) / kPer;
    const uint4* p = reinterpret_cast<const uint4*>(w.p + lo);
    const uint4* q = w.q ? reinterpret_cast<const uint4*>(w.q + lo) : nullptr;
    for (int first = 0; first < n; first += 32 * kTurn) {
      int h = 0, l = 0;
      const int last = min(n, first + 32 * kTurn);
#pragma unroll 4
      for (int i = first + lane; i < last; i += 32) {
        const uint4 a = __ldcg(p + i), b = q ? __ldcg(q + i) : a;
        T x[kPer], y[kPer];
        memcpy(x, &a, 16);
        memcpy(y, &b, 16);
#pragma unroll
        for (int e = 0; e < kPer; ++e) w.add(x[e], y[e], lo + i * kPer + e, h, l);
      }
      sum += ((int64_t)h << 23) + l;
    }
    lo += n * kPer;
  }
  for (int first = lo; first < hi; first += 32 * kFlush) {
    int h = 0, l = 0;
    const int last = min(hi, first + 32 * kFlush);
#pragma unroll 8
    for (int v = first + lane; v < last; v += 32) w.add(w.p[v], w.q ? w.q[v] : w.p[v], v, h, l);
    sum += ((int64_t)h << 23) + l;
  }
  return warp_sum(sum);
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const __grid_constant__ VerifyParams vp) {
  const hsa_verify_args& p = vp.a;
  __shared__ int s_kept, s_without;
  __shared__ int64_t s_piece[kWarps], s_scan[kWarps];    // sums of the warps' pieces; of the warps' parts of one piece
  __shared__ uint64_t s_cta;             // of this CTA's share, which the others read
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ctas = vp.ctas;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas, most = p.nq - 1;
  const int n = p.n_draft ? p.n_draft[b] : most;
  if (n < 0 || n > most) {               // the same in every CTA of the cluster
    if (n != -1 && rank == 0 && tid == 0) flag_status(vp.status, HSA_FLAG_INDEX_RANGE);
    return;
  }
  const T* rows_p = static_cast<const T*>(p.p) + (int64_t)b * p.nq * p.p_stride;
  const T* rows_q = p.q ? static_cast<const T*>(p.q) + (int64_t)b * most * p.q_stride : nullptr;
  // ---------------------------------------------------------------- how many stay
  if (warp == 0) {
    bool turned = false, known = true;
    int x = -1;
    if (lane < n) {
      x = p.drafted[(int64_t)b * most + lane];
      const float u = p.u_accept[(int64_t)b * most + lane];
      known = x >= 0 && x < p.vocabulary;
      turned = true;
      if (known) {
        const float px = __saturatef(value_of(rows_p[lane * p.p_stride + x]));
        const float qx = rows_q ? __saturatef(value_of(rows_q[lane * p.q_stride + x])) : 1.f;
        turned = !((double)u * (double)qx < (double)px);
      }
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
  Weights<T> w{rows_p + kept * p.p_stride, rows_q && kept < n ? rows_q + kept * p.q_stride : nullptr, s_without};
  const int per = ((p.vocabulary + ctas * kWarps - 1) / (ctas * kWarps) + kStep - 1) / kStep * kStep;
  auto begin_of = [&](int piece) { return min(p.vocabulary, (rank * kWarps + piece) * per); };

  // ---------------------------------------------------------------- the sums: of pieces, shares, the row
  uint64_t before = 0, total = 0;        // of the CTAs before this one, of all
  for (int turn = 0;; ++turn) {
    const int64_t sum = sum_piece<T, WIDE>(w, begin_of(warp), begin_of(warp + 1), lane);
    if (lane == 0) s_piece[warp] = sum;
    __syncthreads();
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) mine += (uint64_t)s_piece[i];
    if (ctas > 1) {
      if (tid == 0) s_cta = mine;
      __syncthreads();
      cluster_sync_all();
      before = total = 0;
      for (int c = 0; c < ctas; ++c) {
        const uint64_t x = ld_cluster_u64(cluster_map(smem_u32(&s_cta), c));
        if (c < rank) before += x;
        total += x;
      }
      __syncwarp();
      cluster_arrive();                  // waited for below: until then the others may read this CTA's sum
    } else {
      total = mine;
    }
    if (total || turn) break;
    w.q = nullptr;                       // nothing is left of p: p itself
    w.without = -1;
    if (ctas > 1) cluster_wait();
    __syncthreads();
  }
  // ---------------------------------------------------------------- the piece and the entry that pass the border
  if (total) {
    const uint32_t bits = __float_as_uint(fminf(fmaxf(p.u_sample[b], 0.f), 0x1.fffffep-1f));   // NaN: 0
    const int left = (int)(bits >> 23) - 86;             // 2^(e - 150) in units of 2^-64
    const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u;
    const uint64_t border = __umul64hi(total, left >= 0 ? m << left : left > -24 ? m >> -left : 0ull);
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
  } else if (rank == 0 && tid == 0) {
    p.tokens[(int64_t)b * p.nq + kept] = -1;
    flag_status(vp.status, HSA_FLAG_NO_WEIGHT);
  }
  __syncwarp();
  if (ctas > 1) cluster_wait();
}

template <typename T>
cudaError_t launch(const VerifyParams& p, cudaStream_t s) {
  auto kernel = p.wide ? draft_verify_kernel<T, true> : draft_verify_kernel<T, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.batch * p.ctas);
  cfg.blockDim = dim3(kThreads);
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

}  // namespace

cudaError_t launch_draft_verify(const hsa_verify_args& a, uint32_t* status, cudaStream_t s) {
  VerifyParams p;
  p.a = a;
  p.status = status;
  // as many CTAs to a request as give every SM two, while each has 2,048 entries
  p.ctas = 1;
  while (p.ctas < 8 && (int64_t)p.ctas * a.batch < 2 * kSms && a.vocabulary / p.ctas > 2048) p.ctas *= 2;
  const int size = a.dtype == HSA_F32 ? 4 : 2;
  p.wide = ((reinterpret_cast<uintptr_t>(a.p) | reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)(a.p_stride * size) |
             (uintptr_t)(a.q ? a.q_stride * size : 0)) & 15) == 0;
  switch (a.dtype) {
    case HSA_F32: return launch<float>(p, s);
    case HSA_BF16: return launch<__nv_bfloat16>(p, s);
    default: return launch<__half>(p, s);
  }
}

}  // namespace hsa
