// 4-bit rows of paged caches (HSA_E2M1): where a row's bytes lie, and how 16 values become codes and a scale.
#pragma once

#include "hsa_common.cuh"

namespace hsa {

// Dims 8 c .. 8 c + 7 of a row, its bytes 4 c .. 4 c + 3, lie
//  - in a row of K as two neighbouring pairs of bytes, at four_k_at<D>(c, 0) and four_k_at<D>(c, 1),
//  - in a row of V as single bytes, at four_v_at<D>(c, 0) .. four_v_at<D>(c, 3).
template <int D>
__device__ __forceinline__ int four_k_at(int c, int half) { return D / 8 * (2 * (c & 1) + half) + 2 * (c >> 1); }
template <int D>
__device__ __forceinline__ int four_v_at(int c, int byte) { return D / 16 * (4 * (c & 1) + byte) + (c >> 1); }

// The smallest positive E4M3 value s with 6 s >= amax (448 above 6 * 448), as its byte: the nearest one to amax / 6, or
// the next where that is too small. (amax / 6 in fp32 may be off by 2^-23 of it, far less than a step: only where it
// lies beside the middle of two steps can the rounding go either way, and then the comparison decides.)
__device__ __forceinline__ uint32_t four_scale_for(float amax) {
  uint16_t near;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(near) : "f"(0.f), "f"(amax * (1.f / 6.f)));
  uint32_t byte = max(near & 0x7Fu, 1u);
  if (6.f * e4m3_to_f32(byte) < amax && byte < 0x7Eu) ++byte;
  return byte;
}

// The largest magnitude, NaN if any is
__device__ __forceinline__ float abs_max(float x, float y, float z) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Eight values, in pairs, -> four bytes of E2M1 codes of x / s (nearest even, saturating), -0 as 0. |x| <= 7 s, s > 0. The quotient is
// q = x r with r = 1 / s to a unit in the last place, plus the part of the exact remainder (P. Markstein, 1990): one that
// lies between two codes is exact, and none beside it becomes it, as s has 4 bits and x / s is then more than half a unit away
__device__ __forceinline__ uint32_t four_codes(const uint64_t (&x)[4], float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  const uint64_t rr = f2_pack(r, r), minus = f2_pack(-s, -s);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q = f2_mul(x[i], rr);
    float lo, hi;
    f2_unpack(f2_fma(f2_fma(q, minus, x[i]), rr, q), lo, hi);
    w |= (f32x2_to_e2m1x2(hi, lo) & 0xFFu) << (8 * i);
  }
  const uint32_t m = w & 0x77777777u;    // a sign stays where the magnitude is not 0: then, and only then, m + 7 carries into it
  return w & (0x77777777u | ((m + 0x77777777u) & 0x88888888u));
}

// (x, x) of the low or the high half of an f16 pair times y
__device__ __forceinline__ uint32_t mul_half(uint32_t x, int hi, uint32_t y) {
  const __half2 a = *reinterpret_cast<const __half2*>(&x), b = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hmul2(hi ? __high2half2(a) : __low2half2(a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace hsa
