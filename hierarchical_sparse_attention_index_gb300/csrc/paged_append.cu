// New tokens into the pages of a dense layer's cache with the position rotation on the way (hsa_paged_cache_append), and
// pages back into rows (hsa_paged_cache_read).
//   pos = start[b] + t - cu[b];  pair i of a head of q or k: (x, y) -> (x cos - y sin, x sin + y cos) of the angle pos inv_freq[i];
//   q_out[t] = round(rotated q[t]),  page[table[b][pos / P]][h][pos % P] = round(rotated k[t] or v[t], times 1 / scale).
//
// Bound: every element is read and written once, so HBM decides for prompts, the chain of dependent loads (cu, then
// start and the table, then the stores) for single tokens. A thread's unit is two 16-byte pieces of a head, which
// for rotated halves are the two ends of its 8 pairs, so that nothing is read twice and q may be rotated in
// place. Loads of two units go first; while they fly, a block finds its rows' slots and the sines of
// its rows, once for all heads. The angle is a 64-bit fraction of a turn times the position, whose wrapping product is
// exact (the fraction is not, by up to 2^-64); what is left of a quarter turn goes through sincospif.
// Codes of 4 bits are put in the pool's order in shared memory, so that whole 8-byte pieces are written; warps whose heads
// are q's alone skip that.
// Measured: 65,536 tokens of 32 + 8 + 8 heads of 128 dims, bf16, into E4M3 pages 230 us, 0.94 of the measured copy rate, into bf16 pages 242, 0.98, into
// 4-bit pages 253, 0.83; 16,384 into those 70 us, 0.75 (with the read of their rows 89; with codes for every head, and without
// packed arithmetic, 131). There the schedulers issue in 68 % of the clocks, no unit is above 47 % and HBM at 56: what is left is
// loads, fixed latencies and a block's first barriers, which the 28 warps of an SM do not cover. 64 single tokens 3.4 us (the launch, and loads that
// wait for one another).
// hsa_paged_cache_write of 65,536 tokens of 8 + 8 heads into 4-bit pages 94 us, 0.54 (into bf16 pages 83, 0.95), of 16,384 32 us, 0.40: every warp
// makes codes, 20 instructions to an element (17.5 in the append, on average); issue 74 %, the integer and conversion unit 61 %, HBM 43.
// Back into rows, 8 heads of 128 dims: 262,144 rows from 4-bit pages 215 us, 0.94, from E4M3 238, 1.00, from bf16 308, 1.03; 5,065 rows of
// 4 heads of 64 dims from E4M3 3.0 us.
#include "hsa_dense.h"
#include "hsa_four.cuh"
#include "hsa_rows.cuh"
#include "hsa_softmax.cuh"

namespace hsa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;                // units in flight per thread
constexpr int kMaxRows = 32;             // of a block
constexpr int kMaxPairs = 64;

template <bool BF16>
__device__ __forceinline__ void widen(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = half_at(w[i], 0, BF16);
    x[2 * i + 1] = half_at(w[i], 1, BF16);
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float inv) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
    r[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(r[0], r[1]);
}

// (cos, sin) of pos * turns / 2^64 turns
__device__ __forceinline__ float2 cos_sin(int64_t pos, uint64_t turns) {
  const uint64_t ph = (uint64_t)pos * turns;
  const uint64_t quarter = (ph + (1ull << 61)) >> 62;    // the nearest quarter turn
  float s, c;
  sincospif((float)(int64_t)(ph - (quarter << 62)) * 0x1p-63f, &s, &c);
  const float2 r = (quarter & 1) ? make_float2(-s, c) : make_float2(c, s);
  return (quarter & 2) ? make_float2(-r.x, -r.y) : r;
}
// radians per position as a 64-bit fraction of a turn, cut off below 2^-64. A pair that turns back takes the fraction of its
// magnitude, whose floor leaves an exact rest: 1 - |t| would keep 2^-54 of a turn only
__device__ __forceinline__ uint64_t turns_of(float radians) {
  const double t = fabs((double)radians * 0.15915494309189533577);
  const uint64_t turns = __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
  return radians < 0.f ? 0ull - turns : turns;
}

template <int D, int KV, bool BF16>
__global__ void __launch_bounds__(kThreads, KV == HSA_E2M1 ? 4 : 0) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int kPer = D / 16;           // units per head: pieces cA and cB of its D / 8
  constexpr bool kFour = KV == HSA_E2M1;
  constexpr int kRowBytes = D / 2 + 8;   // of a staged 4-bit row: codes, scales
  __shared__ RowSlots s_rows;
  __shared__ uint64_t s_turns[kMaxPairs];
  __shared__ __align__(16) float2 s_cs[kMaxRows * kMaxPairs];            // (cos, sin) of row r's pairs, from r * pairs on (pair_at)
  __shared__ __align__(16) uint8_t s_four[kFour ? kThreads / kPer * kRowBytes : 16];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int heads = p.heads_q + 2 * p.w.heads;
  const int h0 = blockIdx.y * p.slice, nh = min(p.slice, heads - h0);
  const int64_t t0 = (int64_t)blockIdx.x * p.w.rows_per_block;
  const int n_rows = (int)imin64(p.w.rows_per_block, p.w.n_tokens - t0);
  const int units = n_rows * nh * kPer;
  const int pairs = p.rotary / 2, turned = p.rotary / 16, at0 = p.rotary_at / 8;   // units that rotate, first piece of them
  // Pair i's place: two neighbouring pairs are 16 bytes, which the threads of a head read side by side. A piece has 8 pairs, halves
  // sharing them, or 4
  const bool halves = p.pairs == HSA_ROPE_HALVES;
  const int piece_pairs = halves ? 8 : 4, lines = pairs / piece_pairs;
  auto pair_at = [&](int i) { return 2 * ((i % piece_pairs >> 1) * lines + i / piece_pairs) + (i & 1); };
  // a thread's next unit is kThreads further: no division on the way
  int e = tid, row_at = tid / kPer / nh, head_at = tid / kPer % nh;
  const int row_step = kThreads / kPer / nh, head_step = kThreads / kPer % nh, u = tid % kPer;

  const int after = u - turned, half = kPer - turned;    // of the pieces that do not turn, which go around the others
  const int ca = after < 0 ? at0 + u : (after < at0 ? after : after + 2 * turned);
  const int cb = after < 0 ? at0 + u + turned : (after + half < at0 ? after + half : after + half + 2 * turned);
  for (int base = 0; base < units; base += kThreads * kUnits) {
    uint4 x[kUnits][2];
    int row[kUnits], head[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      row[i] = e < units ? row_at : -1;
      head[i] = h0 + head_at;
      e += kThreads;
      row_at += row_step;
      head_at += head_step;
      if (head_at >= nh) {
        head_at -= nh;
        ++row_at;
      }
      if (row[i] >= 0) {
        const int64_t t = t0 + row[i];
        const int hk = head[i] - p.heads_q, hv = hk - p.w.heads;
        const uint16_t* src = hk < 0 ? p.q + t * p.q_stride + head[i] * D : hv < 0 ? p.w.k + t * p.w.k_stride + hk * D : p.w.v + t * p.w.v_stride + hv * D;
        x[i][0] = *reinterpret_cast<const uint4*>(src + 8 * ca);
        x[i][1] = *reinterpret_cast<const uint4*>(src + 8 * cb);
      } else {
        x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (base == 0) {
      if (tid < pairs) s_turns[tid] = turns_of(p.inv_freq[tid]);
      find_slots(p.w, t0, n_rows, s_rows, h0 == 0 ? HSA_FLAG_WRITE_RANGE : 0u);
      for (int k = tid; k < n_rows * pairs; k += kThreads) {
        const int r = k / pairs, i = k - r * pairs;
        s_cs[r * pairs + pair_at(i)] = cos_sin(s_rows.pos[r], s_turns[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int r = max(row[i], 0), hk = head[i] - p.heads_q, hv = hk - p.w.heads;
      float a[8], b[8];
      widen<BF16>(x[i][0], a);
      widen<BF16>(x[i][1], b);
      if (u < turned && hv < 0) {
        const float4* cs = reinterpret_cast<const float4*>(s_cs + r * pairs) + u;      // (cos, sin) of two pairs
        if (halves) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 y = cs[j * lines];
            const float m = a[2 * j], n = b[2 * j], o = a[2 * j + 1], q = b[2 * j + 1];
            a[2 * j] = fmaf(m, y.x, -(n * y.y));
            b[2 * j] = fmaf(m, y.y, n * y.x);
            a[2 * j + 1] = fmaf(o, y.z, -(q * y.w));
            b[2 * j + 1] = fmaf(o, y.w, q * y.z);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 y = cs[j * lines], z = cs[j * lines + turned];
            const float m = a[4 * j], n = a[4 * j + 1], o = a[4 * j + 2], q = a[4 * j + 3];
            a[4 * j] = fmaf(m, y.x, -(n * y.y));
            a[4 * j + 1] = fmaf(m, y.y, n * y.x);
            a[4 * j + 2] = fmaf(o, y.z, -(q * y.w));
            a[4 * j + 3] = fmaf(o, y.w, q * y.z);
            const float m2 = b[4 * j], n2 = b[4 * j + 1], o2 = b[4 * j + 2], q2 = b[4 * j + 3];
            b[4 * j] = fmaf(m2, z.x, -(n2 * z.y));
            b[4 * j + 1] = fmaf(m2, z.y, n2 * z.x);
            b[4 * j + 2] = fmaf(o2, z.z, -(q2 * z.w));
            b[4 * j + 3] = fmaf(o2, z.w, q2 * z.z);
          }
        }
        x[i][0] = narrow<BF16>(a);
        x[i][1] = narrow<BF16>(b);
      }
      const int64_t slot = row[i] < 0 ? -1 : s_rows.slot[r];
      if (hk < 0) {
        if (row[i] >= 0 && s_rows.real[r]) {
          uint16_t* dst = p.q_out + (t0 + r) * p.out_stride + head[i] * D;
          *reinterpret_cast<uint4*>(dst + 8 * ca) = x[i][0];
          *reinterpret_cast<uint4*>(dst + 8 * cb) = x[i][1];
        }
      } else if (!kFour && slot >= 0) {
        const int64_t at = slot + (int64_t)(hv < 0 ? hk : hv) * p.w.page_size;         // row of the pool
        uint8_t* pool = hv < 0 ? p.w.k_pool : p.w.v_pool;
        if constexpr (KV == HSA_E4M3) {
          const float inv = hv < 0 ? p.w.k_inv : p.w.v_inv;
          *reinterpret_cast<uint2*>(pool + at * D + 8 * ca) = e4m3x8(a, inv);
          *reinterpret_cast<uint2*>(pool + at * D + 8 * cb) = e4m3x8(b, inv);
        } else {
          *reinterpret_cast<uint4*>(pool + (at * D + 8 * ca) * 2) = x[i][0];
          *reinterpret_cast<uint4*>(pool + (at * D + 8 * cb) * 2) = x[i][1];
        }
      }
      if (kFour && __any_sync(0xffffffffu, hk >= 0 && slot >= 0)) {      // most warps have heads of q alone, or none
        // codes of the pool's row, put in its order in shared memory. Two neighbouring lanes hold a group's 16 dims
        const float inv = hv < 0 ? p.w.k_inv : p.w.v_inv;
        uint8_t* mine = s_four + tid / kPer * kRowBytes;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          uint64_t y[4];
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* from = o ? b : a;
            y[j] = f2_mul(f2_pack(from[2 * j], from[2 * j + 1]), f2_pack(inv, inv));
            float lo, hi;
            f2_unpack(y[j], lo, hi);
            amax = abs_max(amax, lo, hi);
          }
          amax = abs_max(amax, __shfl_xor_sync(0xffffffffu, amax, 1), 0.f);
          const uint32_t byte = amax != amax ? 0x7Fu : four_scale_for(amax);
          const int c = o ? cb : ca;
          if (byte == 0x7Eu)             // the largest scale may be too small
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float lo, hi;
              f2_unpack(y[j], lo, hi);
              y[j] = f2_pack(fminf(fmaxf(lo, -3136.f), 3136.f), fminf(fmaxf(hi, -3136.f), 3136.f));
            }
          const uint32_t w = byte == 0x7Fu ? 0u : four_codes(y, e4m3_to_f32(byte));
          if (hv < 0) {
            *reinterpret_cast<uint16_t*>(mine + four_k_at<D>(c, 0)) = (uint16_t)w;
            *reinterpret_cast<uint16_t*>(mine + four_k_at<D>(c, 1)) = (uint16_t)(w >> 16);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) mine[four_v_at<D>(c, j)] = (uint8_t)(w >> (8 * j));
          }
          if (!(c & 1)) mine[D / 2 + (c >> 1)] = (uint8_t)byte;
        }
        __syncwarp();
        if (hk >= 0 && slot >= 0) {
          const int64_t at = slot + (int64_t)(hv < 0 ? hk : hv) * p.w.page_size;
          uint8_t* pool = hv < 0 ? p.w.k_pool : p.w.v_pool;
          uint8_t* scales = hv < 0 ? p.w.k_s : p.w.v_s;
          const int part = lane % kPer;
          *reinterpret_cast<uint2*>(pool + at * (D / 2) + 8 * part) = *reinterpret_cast<const uint2*>(mine + 8 * part);
          if (part == 0) {
            if constexpr (D == 128)
              *reinterpret_cast<uint2*>(scales + at * (D / 16)) = *reinterpret_cast<const uint2*>(mine + D / 2);
            else
              *reinterpret_cast<uint32_t*>(scales + at * (D / 16)) = *reinterpret_cast<const uint32_t*>(mine + D / 2);
          }
        }
        __syncwarp();
      }
    }
  }
}

// ------------------------------------------------------------------ pages back into rows
constexpr int kReadPieces = 4;           // 16-byte pieces of k, and as many of v, in flight per thread

template <int D, int KV, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  constexpr int kPer = D / 8;            // 16-byte pieces of a head's row
  __shared__ RowSlots s_rows;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, per_row = p.w.heads * kPer;
  const int64_t t0 = (int64_t)blockIdx.x * p.w.rows_per_block;
  const int n_rows = (int)imin64(p.w.rows_per_block, p.w.n_tokens - t0);
  find_slots(p.w, t0, n_rows, s_rows, HSA_FLAG_INDEX_RANGE);
  const int pieces = n_rows * per_row;
  for (int base = 0; base < pieces; base += kThreads * kReadPieces) {
    uint4 x[2][kReadPieces];
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int e = base + i * kThreads + tid, r = e / per_row, rest = e - r * per_row, h = rest / kPer, c = rest % kPer;
      const int64_t slot = e < pieces ? s_rows.slot[r] : -1;
      if (slot < 0) continue;
      const int64_t at = slot + (int64_t)h * p.w.page_size;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* pool = kv ? p.w.v_pool : p.w.k_pool;
        if constexpr (KV == HSA_E4M3) {
          const uint2 w = *reinterpret_cast<const uint2*>(pool + at * D + 8 * c);
          x[kv][i].x = w.x;
          x[kv][i].y = w.y;
        } else {
          x[kv][i] = *reinterpret_cast<const uint4*>(pool + (at * D + 8 * c) * 2);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int e = base + i * kThreads + tid, r = e / per_row, rest = e - r * per_row;
      if (e >= pieces || s_rows.slot[r] < 0) continue;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint4 y = x[kv][i];
        const float scale = kv ? p.v_scale : p.k_scale;
        if constexpr (KV == HSA_E4M3) {
          const uint32_t w[2] = {y.x, y.y};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t f = e4m3x2_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
            o[j] = pack2<BF16>(half_at(f, 0, false) * scale, half_at(f, 1, false) * scale);
          }
          y = make_uint4(o[0], o[1], o[2], o[3]);
        }
        uint16_t* dst = (kv ? p.v + (t0 + r) * p.w.v_stride : p.k + (t0 + r) * p.w.k_stride) + 8 * rest;
        __stcs(reinterpret_cast<uint4*>(dst), y);
      }
    }
  }
}

// 4-bit pages: a thread reads 8 bytes of a row of K, and of V, in the pages' order, and writes their 16 dims where they belong: four
// (two) neighbouring ones of a scale's group at a time, which the threads of a row make up to whole 32-byte sectors
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_read_four_kernel(const __grid_constant__ PagedReadParams p) {
  constexpr int kPer = D / 16;           // 8-byte pieces of a head's row
  __shared__ RowSlots s_rows;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, per_row = p.w.heads * kPer, part = tid % kPer;
  const int64_t t0 = (int64_t)blockIdx.x * p.w.rows_per_block;
  const int n_rows = (int)imin64(p.w.rows_per_block, p.w.n_tokens - t0);
  find_slots(p.w, t0, n_rows, s_rows, HSA_FLAG_INDEX_RANGE);
  const int pieces = n_rows * per_row;
  // two values of a code byte, times the scale of its group (exact in f16) and of the pool
  auto values = [](uint32_t f16x2, float scale) { return pack2<BF16>(half_at(f16x2, 0, false) * scale, half_at(f16x2, 1, false) * scale); };
  for (int base = 0; base < pieces; base += kThreads * kReadPieces) {
    uint2 k[kReadPieces], v[kReadPieces], ks[kReadPieces], vs[kReadPieces];
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int e = base + i * kThreads + tid, r = e / per_row, h = (e - r * per_row) / kPer;
      const int64_t slot = e < pieces ? s_rows.slot[r] : -1;
      if (slot < 0) continue;
      const int64_t at = slot + (int64_t)h * p.w.page_size;
      k[i] = *reinterpret_cast<const uint2*>(p.w.k_pool + at * (D / 2) + 8 * part);
      v[i] = *reinterpret_cast<const uint2*>(p.w.v_pool + at * (D / 2) + 8 * part);
      if constexpr (D == 128) {
        ks[i] = *reinterpret_cast<const uint2*>(p.w.k_s + at * kPer);
        vs[i] = *reinterpret_cast<const uint2*>(p.w.v_s + at * kPer);
      } else {
        ks[i] = make_uint2(*reinterpret_cast<const uint32_t*>(p.w.k_s + at * kPer), 0u);
        vs[i] = make_uint2(*reinterpret_cast<const uint32_t*>(p.w.v_s + at * kPer), 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int e = base + i * kThreads + tid, r = e / per_row, h = (e - r * per_row) / kPer;
      if (e >= pieces || s_rows.slot[r] < 0) continue;
      uint16_t* to_k = p.k + (t0 + r) * p.w.k_stride + h * D;
      uint16_t* to_v = p.v + (t0 + r) * p.w.v_stride + h * D;
      // K: bytes 2 j, 2 j + 1 are dims 4 t .. 4 t + 3 of group s0 + j
      const int t = D == 128 ? part >> 1 : part, s0 = D == 128 ? 4 * (part & 1) : 0;
      const uint32_t kw[2] = {k[i].x, k[i].y}, vw[2] = {v[i].x, v[i].y};
      const uint32_t kc = s0 ? ks[i].y : ks[i].x;        // their scales
      const uint32_t f0 = e4m3x2_to_f16x2((uint16_t)(kc & 0xFFFFu)), f1 = e4m3x2_to_f16x2((uint16_t)(kc >> 16));
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t x[4];
        e2m1x8_to_f16x2x4(kw[w], x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          __stcs(reinterpret_cast<uint2*>(to_k + 16 * (s0 + 2 * w + j) + 4 * t),
                 make_uint2(values(mul_half(w ? f1 : f0, j, x[2 * j]), p.k_scale), values(mul_half(w ? f1 : f0, j, x[2 * j + 1]), p.k_scale)));
      }
      // V, 128 dims: byte s is dims 2 r, 2 r + 1 of group s, r = part; 64 dims: bytes s and 4 + s those of r = 2 part and 2 part + 1
      uint32_t x[2][4];
#pragma unroll
      for (int w = 0; w < 2; ++w) e2m1x8_to_f16x2x4(vw[w], x[w][0], x[w][1], x[w][2], x[w][3]);
      if constexpr (D == 128) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t vc = w ? vs[i].y : vs[i].x;
          const uint32_t g0 = e4m3x2_to_f16x2((uint16_t)(vc & 0xFFFFu)), g1 = e4m3x2_to_f16x2((uint16_t)(vc >> 16));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            __stcs(reinterpret_cast<uint32_t*>(to_v + 16 * (4 * w + j) + 2 * part), values(mul_half(j < 2 ? g0 : g1, j & 1, x[w][j]), p.v_scale));
        }
      } else {
        const uint32_t g0 = e4m3x2_to_f16x2((uint16_t)(vs[i].x & 0xFFFFu)), g1 = e4m3x2_to_f16x2((uint16_t)(vs[i].x >> 16));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __stcs(reinterpret_cast<uint2*>(to_v + 16 * j + 4 * part), make_uint2(values(mul_half(j < 2 ? g0 : g1, j & 1, x[0][j]), p.v_scale),
                                                                                values(mul_half(j < 2 ? g0 : g1, j & 1, x[1][j]), p.v_scale)));
      }
    }
  }
}

template <int D, int KV, bool BF16>
cudaError_t append(PagedAppendParams p, cudaStream_t s) {
  constexpr int kPer = D / 16;
  const int64_t heads = (int64_t)p.heads_q + 2 * p.w.heads, row = heads * kPer;        // units per token
  // whole rows, about twelve units to a thread (65,536 tokens of 48 heads into E4M3 pages, 6, 8, 12, 16, 24, 32 units: 238, 240, 230, 236,
  // 233, 241 us, into bf16 243, 245, 242, 248, 246, 254); fewer rows, then slices of a row's heads, while there are SMs without a block
  const int64_t most = imin64(kMaxRows, imax64(1, 12 * kThreads / row));
  p.w.rows_per_block = (int32_t)imax64(1, imin64(most, (p.w.n_tokens + 2 * kSms - 1) / (2 * kSms)));
  const int64_t blocks = (p.w.n_tokens + p.w.rows_per_block - 1) / p.w.rows_per_block;
  int64_t slices = imin64((2 * kSms + blocks - 1) / blocks, (row + kThreads - 1) / kThreads);
  p.slice = (int32_t)((heads + slices - 1) / slices);
  slices = (heads + p.slice - 1) / p.slice;
  return launch_pdl(paged_append_kernel<D, KV, BF16>, dim3((unsigned)blocks, (unsigned)slices), dim3(kThreads), 0, s, p);
}
template <int D, int KV, bool BF16>
cudaError_t read(PagedReadParams p, cudaStream_t s) {
  constexpr bool kFour = KV == HSA_E2M1;
  const int64_t row = (int64_t)p.w.heads * (D / (kFour ? 16 : 8));       // pieces of a row
  const int64_t most = imin64(kMaxRows, imax64(1, kThreads * kReadPieces / row)), least = imin64(kMaxRows, imax64(1, kThreads / row));
  // Fewer rows than that while every SM does not have two blocks; of 4-bit pages four, which is what it holds. With two and four: 10,500
  // rows of 4 heads of 128 dims from 4-bit pages 8.3 and 5.8 us, 5,600 rows of 4 heads of 64 dims from E4M3 pages 3.0 and 3.9
  constexpr int64_t kBlocks = (kFour ? 4 : 2) * kSms;
  p.w.rows_per_block = (int32_t)imin64(most, imax64(least, (p.w.n_tokens + kBlocks - 1) / kBlocks));
  const int64_t blocks = (p.w.n_tokens + p.w.rows_per_block - 1) / p.w.rows_per_block;
  if constexpr (kFour)
    return launch_pdl(paged_read_four_kernel<D, BF16>, dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
  else
    return launch_pdl(paged_read_kernel<D, KV, BF16>, dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
}

// the kernel of this head size, cache type and 16-bit type
#define HSA_BY_TYPE(call, head_dim, kv, bf16, ...)                                                        \
  switch (kv) {                                                                                           \
    case HSA_BF16: return head_dim == 128 ? call<128, HSA_BF16, true>(__VA_ARGS__) : call<64, HSA_BF16, true>(__VA_ARGS__);   \
    case HSA_F16: return head_dim == 128 ? call<128, HSA_F16, false>(__VA_ARGS__) : call<64, HSA_F16, false>(__VA_ARGS__);    \
    case HSA_E4M3:                                                                                        \
      if (bf16) return head_dim == 128 ? call<128, HSA_E4M3, true>(__VA_ARGS__) : call<64, HSA_E4M3, true>(__VA_ARGS__);      \
      return head_dim == 128 ? call<128, HSA_E4M3, false>(__VA_ARGS__) : call<64, HSA_E4M3, false>(__VA_ARGS__);              \
    default:                                                                                              \
      if (bf16) return head_dim == 128 ? call<128, HSA_E2M1, true>(__VA_ARGS__) : call<64, HSA_E2M1, true>(__VA_ARGS__);      \
      return head_dim == 128 ? call<128, HSA_E2M1, false>(__VA_ARGS__) : call<64, HSA_E2M1, false>(__VA_ARGS__);              \
  }

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int32_t kv_dtype, cudaStream_t s) {
  HSA_BY_TYPE(append, p.w.head_dim, kv_dtype, p.w.bf16, p, s)
}
cudaError_t launch_paged_read(const PagedReadParams& p, int32_t kv_dtype, cudaStream_t s) {
  HSA_BY_TYPE(read, p.w.head_dim, kv_dtype, p.w.bf16, p, s)
}

}  // namespace hsa
