// Pieces shared by the dense attention kernels on tcgen05: products issued from warp-uniform code,
// tensor-map copies, waits that sleep, and the softmax of one key tile with a query row per thread.
#pragma once

#include <cuda.h>

#include "hsa_common.cuh"
#include "hsa_softmax.cuh"
#include "hsa_tc.cuh"

namespace hsa {

// mbar_wait with a suspend hint: a waiting warp sleeps in the barrier unit instead of coming back to
// ask, which would take shared-memory cycles from the products (4 % of a long prompt's time)
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return done != 0;
}
// Each lane has its own limit: a warp votes on the outcome before it goes on.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_sleep(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_sleep(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// A kernel that hands registers from group to group (setmaxnreg) waits without a limit for more than its launch
// holds, so what the compiler gave it is looked at before the first launch.
template <class Kernel>
bool launches_with(Kernel kernel, int regs) {
  cudaFuncAttributes attr;
  return cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(kernel)) == cudaSuccess && attr.numRegs >= regs;
}

// For a CTA's own copies and products in flight, before it ends: nothing may still write into its shared or
// tensor memory then, however short the caller's limit is
__device__ __forceinline__ bool drain_bar(uint32_t bar, uint32_t parity) { return wait_bar(bar, parity, kWaitLimitNs); }
// Whether the phase is complete, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Products and commits issued by one lane (`one` is nonzero in it) of a warp that stays together: in
// code that the whole warp runs, descriptors live in uniform registers, where these instructions
// take them from; under a branch of the one lane every product would first have to move its four
// there (88 clocks a product instead of 64 and less)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(one));
  return one;
}
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; setp.ne.b32 p, %4, 0; setp.ne.b32 e, %5, 0;\n"
      "  @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one));
}
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, e; setp.ne.b32 p, %4, 0; setp.ne.b32 e, %5, 0;\n"
      "  @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(one));
}
__device__ __forceinline__ void umma_commit_one(uint32_t one, uint32_t bar) {
  asm volatile(
      "{ .reg .pred e; setp.ne.b32 e, %1, 0;\n"
      "  @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Cluster launch control: ask the launcher for a block of this grid that has not started. The
// 16-byte answer lands in shared memory; it holds the block's index, or nothing if none is left.
__device__ __forceinline__ void next_block_ask(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool next_block_take(uint32_t answer, uint32_t& block) {
  uint32_t got;
  asm volatile(
      "{ .reg .pred p; .reg .b128 a; ld.shared.b128 a, [%2];\n"
      "  clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
      "  selp.u32 %0, 1, 0, p; mov.u32 %1, 0;\n"
      "  @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a; }"
      : "=r"(got), "=r"(block)
      : "r"(answer)
      : "memory");
  return got != 0;
}

// Tensor-map copies from code that the whole warp runs (`one` is nonzero in the lane that issues)
__device__ __forceinline__ void tma_4d_one(uint32_t one, uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %7, 0;\n"
      "@p cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6]; }" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "r"(one)
      : "memory");
}

__device__ __forceinline__ void tma_3d_one(uint32_t one, uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n"
      "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5]; }" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one)
      : "memory");
}

// 32 bytes of 16-bit values, 32-byte aligned
__device__ __forceinline__ void st_global_256(void* at, const uint32_t* y) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]),
               "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
#define TMEM_ST8(taddr, r)                                                                                      \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),  \
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)                     \
               : "memory")
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// -inf where c < lo or c >= hi: by bits, so that a column costs a predicate move and a select instead of
// two comparisons
__device__ __forceinline__ void mask_row(uint32_t (&s)[2][32], int lo, int hi) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int h = min(max(hi - 32 * c, 0), 32), l = min(max(lo - 32 * c, 0), 32);
    const uint32_t below_h = h == 32 ? 0xFFFFFFFFu : (1u << h) - 1u, below_l = l == 32 ? 0xFFFFFFFFu : (1u << l) - 1u;
    const uint32_t keep = below_h & ~below_l;
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(keep & (1u << e))) s[c][e] = 0xFF800000u;
  }
}

// The softmax of 64 keys, one query row per thread: S in the tensor memory columns at .. at + 63 is
// taken into the running maximum m (in units of S) and sum l, and P = 2^((S - m) scale + kLift), rounded to the
// operand type, goes into its first 32 columns. `mask(s)` writes -inf where a row does not see a key;
// `sees`: this thread's row sees a key of the tile. The maximum is only raised where a logit passes
// it by 2^8 in some row of the warp; O (D columns at tO) is then rescaled, after wait_o() if `later`
// (an earlier tile has gone into it).
template <int D, bool BF16, typename Mask, typename WaitO>
__device__ __forceinline__ void softmax_tile(uint32_t at, uint32_t tO, bool sees, float scale, float& m, float& l, bool later,
                                             Mask&& mask, WaitO&& wait_o) {
  uint32_t s[2][32];
#pragma unroll
  for (int c = 0; c < 2; ++c) TMEM_LD32(at + 32 * c, s[c]);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 2; ++c) tmem_regs_ready(s[c]);
  mask(s);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 16; c += 2)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      mx[u] = max3(mx[u], __uint_as_float(s[u >> 1][16 * (u & 1) + c]), __uint_as_float(s[u >> 1][16 * (u & 1) + c + 1]));
  const float top = sees ? max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) : -INFINITY;
  if (__any_sync(0xffffffffu, (top - m) * scale > kRaise)) {     // also with m = -inf; not with top = -inf
    const float mn = fmaxf(m, top);
    const float f = mn == -INFINITY ? 1.f : ex2_ftz((m - mn) * scale);   // m = -inf before: 0, on sums that are 0
    m = mn;
    l *= f;
    if (later) {
      wait_o();
#pragma unroll 1
      for (int c = 0; c < D / 8; ++c) {  // 8 columns at a time: the row of S stays in registers
        uint32_t o[8];
        TMEM_LD8(tO + 8 * c, o);
        tmem_wait_ld();
        tmem_regs_ready(o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        TMEM_ST8(tO + 8 * c, o);
      }
    }
  }
  const float mu = m == -INFINITY ? 0.f : fmaf(m, scale, -kLift<BF16>);
  const uint64_t nmu2 = f2_pack(-mu, -mu), scale2 = f2_pack(scale, scale);
  uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {          // 16 keys at a time, so that P takes few registers beside S
    uint32_t pk[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int e = 16 * q + 2 * c;
      float z0, z1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1])), scale2, nmu2), z0, z1);
      const float p0 = ex2_ftz(z0), p1 = ex2_ftz(z1);
      if (c & 1)
        sum1 = f2_add(sum1, f2_pack(p0, p1));
      else
        sum0 = f2_add(sum0, f2_pack(p0, p1));
      pk[c] = pack2<BF16>(p0, p1);
    }
    TMEM_ST8(at + 8 * q, pk);
  }
  tmem_wait_st();
  tc_fence_before();
  float a, b;
  f2_unpack(f2_add(sum0, sum1), a, b);
  l += a + b;
}

}  // namespace hsa
