// The numbers of the dense attention kernels' softmax, and the rounding of their weights and results.
#pragma once

#include "hsa_common.cuh"

namespace hsa {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.f;            // log2 of how far a logit may pass the running maximum
// Weights are 2^(x - m + kLift<BF16>). f16 holds full steps down to 2^-14 only, and keys that are 2^-17 of the largest may be
// many: its weights take the room that kRaise leaves above (2^15 of 65,504). The factor is in the sums as well.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace hsa
