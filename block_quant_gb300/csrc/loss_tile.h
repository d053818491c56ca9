// What a loss takes from a tile of logits while it is in registers: each row's softmax
// statistics, or the values of its probabilities.
//
// The statistics of a set of logits are its maximum m and s = the sum of exp(z - m) over all
// but one logit that attains m: the log of their sum is m + log1p(s), and a logit that
// is the maximum has the log-probability -log1p(s), which keeps its relative precision however near
// to 0 it is (with the maximum in the sum it would be lost beside its 1).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_codes.h"

namespace bq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoTarget = -INFINITY;  // in the place of a row's log-sum: the row's values are 0
// Probabilities (and their differences from a target's weight, in [-1, 1]) are held as fp16 times
// 2^14: eleven bits down to 2^-28, and room to 4 where the forward's sum and these differ.
constexpr int kProbBits = 14;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct RowStats {
  float m, s;
  int at;  // where the maximum is
};

// statistics of two sets
__device__ __forceinline__ RowStats joined(RowStats a, RowStats b) {
  const bool swap = b.m > a.m;
  const RowStats hi = swap ? b : a, lo = swap ? a : b;
  const float f = lo.m == hi.m ? 1.f : ex2((lo.m - hi.m) * kLog2e);
  return {hi.m, fmaf(lo.s + 1.f, f, hi.s), lo.m == hi.m ? min(a.at, b.at) : hi.at};
}

// 2^kProbBits exp(z - lse), 0 in a row without a target
__device__ __forceinline__ float scaled_prob(float z, float lse) {
  return lse == kNoTarget ? 0.f : ex2(fmaf(z - lse, kLog2e, float(kProbBits)));
}

// 2^kProbBits (p - 1) of a class whose loss is -log p, precise where p is near 1
__device__ __forceinline__ float scaled_rest(float loss) { return float(1 << kProbBits) * expm1f(-loss); }

// of a lane's row: N logits' products, of which the first `cols` count
template <int N>
__device__ __forceinline__ void lane_stats(float* z, int cols, float zscale, bool on, float2* stats, uint8_t* at) {
#pragma unroll
  for (int j = 0; j < N; ++j) z[j] *= zscale;
  if (cols < N)
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j >= cols) z[j] = -INFINITY;
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (a NaN is in s)
#pragma unroll
  for (int j = 0; j < N; ++j) m4[j & 3] = fmaxf(m4[j & 3], z[j]);
  const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  float s[2] = {0.f, 0.f};
  int count = -1, where = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float e = ex2((z[j] - m) * kLog2e);
    if (z[j] == m)
      ++count, where = j;
    else
      s[j & 1] += e;
  }
  if (on) {
    *stats = make_float2(m, s[0] + s[1] + float(count));
    *at = uint8_t(where);
  }
}

// A row's listed words in a part of the vocabulary, as one word: the place of the first in the row's list (11 bits),
// their count (5 bits, 31 for that many or more) and the first entry (16: place among the row's words << 6 | column).
__host__ __device__ constexpr uint32_t words_record(uint32_t start, uint32_t count, uint32_t first) {
  return start | (count < 31 ? count : 31u) << 11 | first << 16;
}

// The logits z of a lane's row's listed words, by their record; `next` is the record of the row's next part.  (Registers have
// no index: the lanes' logits go through 2 KB of shared memory of the warp's own, 16 columns at a time, 16-byte word c
// of lane l at c ^ ((l >> 1) & 3) of its 64 bytes, which keeps the banks apart.)
template <int N>
__device__ __forceinline__ void lane_picks(const float* z, uint32_t record, const uint32_t* next, const uint16_t* words,
                                           float* picked, uint32_t box, int lane) {
  uint32_t at = record & 0x7FFu, left = record >> 11 & 31u, entry = record >> 16;
  if (!__any_sync(0xFFFFFFFFu, left > 0)) return;
  if (left == 31u) left = (__ldcg(next) & 0x7FFu) - at;
  const uint32_t mine = box + 64u * uint32_t(lane), turn = uint32_t(lane >> 1) & 3u;
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += 16) {
    const bool here = left > 0 && (entry & 63u) < uint32_t(c0 + 16);
    if (!__any_sync(0xFFFFFFFFu, here)) continue;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((c ^ turn) << 4)), "f"(z[c0 + 4 * c]),
                   "f"(z[c0 + 4 * c + 1]), "f"(z[c0 + 4 * c + 2]), "f"(z[c0 + 4 * c + 3])
                   : "memory");
    while (left > 0 && (entry & 63u) < uint32_t(c0 + 16)) {  // (its own bytes: no other lane's)
      const uint32_t col = entry & 15u;
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(mine + (((col >> 2) ^ turn) << 4) + 4u * (col & 3u)) : "memory");
      picked[entry >> 6] = v;
      if (--left > 0) entry = __ldcg(words + ++at);
    }
  }
  __syncwarp();
}

// of a warp's row: the products of columns lane + 32 j < cols, j < J
template <int J>
__device__ __forceinline__ void row_stats(const float* v, int cols, float zscale, int lane, float2* stats, uint8_t* at) {
  float z[J], m = -INFINITY, s = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    z[j] = lane + 32 * j < cols ? v[j] * zscale : -INFINITY;
    m = fmaxf(m, z[j]);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  int count = 0, where = 255;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (z[j] == m)
      ++count, where = min(where, lane + 32 * j);
    else
      s += ex2((z[j] - m) * kLog2e);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  where = __reduce_min_sync(0xFFFFFFFFu, where);
  if (lane == 0) {
    *stats = make_float2(m, s + float(count - 1));
    *at = uint8_t(where);
  }
}

// z: a lane's row of products, of which the first `cols` count, becomes its scaled probabilities
template <int N>
__device__ __forceinline__ void lane_probs(float* z, int cols, float zscale, float lse) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float p = ex2(fmaf(z[j] * zscale - lse, kLog2e, float(kProbBits)));
    z[j] = lse == kNoTarget || j >= cols ? 0.f : p;
  }
}

}  // namespace bq
