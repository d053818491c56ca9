// Row-wise operators of a layer around the DBuffer step on GB300 (sm_103a):
//   k_embed          rows of the token table (bf16, or E4M3 codes with 128x128
//                    tile scales as the AllGather leaves them) times a factor
//   k_embed_chunks,  stable sort of a batch's tokens by id; zeros into the gradient
//   k_embed_place, k_embed_sort
//   k_embed_rows,    the table's gradient: rows of dY summed over equal ids
//   k_embed_join, k_embed_few
//   k_norm*          residual addition, root-mean-square norm, E4M3 codes with
//                    one scale per 128 values of a row (also without the norm:
//                    the row quantiser)
//   k_norm_grad*     the norm's gradients
// All are bound by memory: each reads its inputs once and writes its outputs once.
#include <algorithm>
#include <string>

#include "bq_internal.h"
#include "fp8_codes.h"
#include "once.h"
#include "pdl.h"
#include "row_ops.h"
#include "umma_ptx.h"

namespace bq {
namespace {

int check(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BQ_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return BQ_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// eight bf16 of one 16-byte word
__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// eight E4M3 codes; the half-precision value of every code is exact
__device__ __forceinline__ void decode8(const uint2& w, float* v) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(u[i] >> (16 * j)), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[4 * i + 2 * j] = f.x;
      v[4 * i + 2 * j + 1] = f.y;
    }
}

__device__ __forceinline__ float decode1(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3)));
}

// a NaN among the operands gives NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// ---------------------------------------------------------------- a warp's 256 columns
// Every kernel here gives a warp 256 consecutive columns of a row, eight values a
// lane.  VEC: lane l holds columns 8l .. 8l+7 (16-byte accesses: the pointer, the
// pitch and the width must be multiples of eight values).  Otherwise value e of
// lane l is column 32e + l (2- or 4-byte accesses, still consecutive over the
// lanes): any pointer, pitch and width.
constexpr int kSpan = 256;

template <bool VEC>
__device__ __forceinline__ int column(int lane, int e) {
  return VEC ? 8 * lane + e : 32 * e + lane;
}

// columns c0 + column(lane, e) of a row; those at or past `cols` read as 0
template <bool VEC>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* row, int c0, int cols, int lane, float* v) {
  if (VEC) {
    const int c = c0 + 8 * lane;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (c < cols) w = *reinterpret_cast<const uint4*>(row + c);
    unpack8(w, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      v[e] = c < cols ? __bfloat162float(row[c]) : 0.f;
    }
  }
}

// the same, eight bf16 packed as loaded
template <bool VEC>
__device__ __forceinline__ uint4 load_packed(const __nv_bfloat16* row, int c0, int cols, int lane) {
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (VEC) {
    const int c = c0 + 8 * lane;
    if (c < cols) w = *reinterpret_cast<const uint4*>(row + c);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      u[e] = c < cols ? uint32_t(__bfloat16_as_ushort(row[c])) : 0u;
    }
    w = make_uint4(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
  }
  return w;
}

// Eight consecutive columns a lane (c0 + 8 lane ..) of a row at any 2-byte alignment: the
// aligned 16-byte words that hold them, shifted.  Every word read holds some of the row,
// so it lies in the row's allocation.
__device__ __forceinline__ uint4 load_shifted(const __nv_bfloat16* row, int c0, int cols, int lane) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(row + c0), end = reinterpret_cast<uintptr_t>(row + cols);
  const uint4* p = reinterpret_cast<const uint4*>(a & ~uintptr_t(15));
  const int m = int(a & 15) >> 1;  // elements to drop: the same in every lane
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (reinterpret_cast<uintptr_t>(p + lane) < end) w = __ldg(p + lane);
  if (m == 0) {
    // (elements past the row are masked below)
  } else {
    uint4 n = make_uint4(__shfl_down_sync(0xFFFFFFFFu, w.x, 1), __shfl_down_sync(0xFFFFFFFFu, w.y, 1),
                         __shfl_down_sync(0xFFFFFFFFu, w.z, 1), __shfl_down_sync(0xFFFFFFFFu, w.w, 1));
    if (lane == 31) {
      n = make_uint4(0u, 0u, 0u, 0u);
      if (reinterpret_cast<uintptr_t>(p + 32) < end) n = __ldg(p + 32);
    }
    uint32_t u[8] = {w.x, w.y, w.z, w.w, n.x, n.y, n.z, n.w};
    if (m & 4) {
#pragma unroll
      for (int i = 0; i < 6; ++i) u[i] = u[i + 2 < 8 ? i + 2 : 7];
    }
    if (m & 2) {
#pragma unroll
      for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
    }
    if (m & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], 16);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  const int left = cols - c0 - 8 * lane;  // of this lane's columns inside the row
  if (left < 8) {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = left >= 2 * i + 2 ? u[i] : left == 2 * i + 1 ? u[i] & 0xFFFFu : 0u;
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  return w;
}

template <bool VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* row, int c0, int cols, int lane, const float* v) {
  if (VEC) {
    const int c = c0 + 8 * lane;
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = pack8(v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      if (c < cols) row[c] = __float2bfloat16_rn(v[e]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void load_f32(const float* row, int c0, int cols, int lane, float* v) {
  if (VEC) {
    const int c = c0 + 8 * lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c < cols) {
      a = *reinterpret_cast<const float4*>(row + c);
      b = *reinterpret_cast<const float4*>(row + c + 4);
    }
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      v[e] = c < cols ? row[c] : 0.f;
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_f32(float* row, int c0, int cols, int lane, const float* v) {
  if (VEC) {
    const int c = c0 + 8 * lane;
    if (c < cols) {
      *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      if (c < cols) row[c] = v[e];
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void load_row(const float* row, int c0, int cols, int lane, float* v) {
  load_f32<VEC>(row, c0, cols, lane, v);
}
template <bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int c0, int cols, int lane, float* v) {
  load_bf16<VEC>(row, c0, cols, lane, v);
}
template <bool VEC>
__device__ __forceinline__ void store_row(float* row, int c0, int cols, int lane, const float* v) {
  store_f32<VEC>(row, c0, cols, lane, v);
}
template <bool VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int c0, int cols, int lane, const float* v) {
  store_bf16<VEC>(row, c0, cols, lane, v);
}

// E4M3 codes of a warp's 256 columns (two groups of 128) and the groups' scales:
// a = max |y|, s = a / 448 (the stored scale), code = e4m3(y * (448 / a)), the rule
// of the FP8 parameter tiles.  A NaN reaches its group's scale.
template <bool VEC>
__device__ __forceinline__ void quant_span(const float* y, int c0, int cols, int lane, uint8_t* codes, float* scale,
                                           int64_t ld_scale) {
  if (VEC) {  // lanes 0-15 hold the first group, 16-31 the second
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) a = max3(a, fabsf(y[e]), fabsf(y[e + 1]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    const QScale q = qscale(__float_as_uint(a), 448.f);
    const int c = c0 + 8 * lane;
    if (c < cols) {
      *reinterpret_cast<uint2*>(codes + c) = codes_e4m3(y, q);
      if ((lane & 15) == 0) scale[int64_t(c >> 7) * ld_scale] = q.s;
    }
  } else {  // values 0-3 of every lane belong to the first group, 4-7 to the second
    float a0 = max3(max_nan(fabsf(y[0]), fabsf(y[1])), fabsf(y[2]), fabsf(y[3]));
    float a1 = max3(max_nan(fabsf(y[4]), fabsf(y[5])), fabsf(y[6]), fabsf(y[7]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      a0 = max_nan(a0, __shfl_xor_sync(0xFFFFFFFFu, a0, o));
      a1 = max_nan(a1, __shfl_xor_sync(0xFFFFFFFFu, a1, o));
    }
    const QScale q0 = qscale(__float_as_uint(a0), 448.f), q1 = qscale(__float_as_uint(a1), 448.f);
    const uint2 w0 = codes_e4m3(y, q0), w1 = codes_e4m3(y, q1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + 32 * e + lane;
      const uint32_t w = e < 4 ? w0.x : w1.y;
      if (c < cols) codes[c] = uint8_t(w >> (8 * (e & 3)));
    }
    if (lane == 0 && c0 < cols) scale[int64_t(c0 >> 7) * ld_scale] = q0.s;
    if (lane == 0 && c0 + 128 < cols) scale[int64_t((c0 >> 7) + 1) * ld_scale] = q1.s;
  }
}

// s = a / 448 rounded to nearest (Markstein 1990: a quotient from the rounded reciprocal
// and one exact residual is the rounded quotient), for 2^-100 <= a < infinity
__device__ __forceinline__ float over_448(float a) {
  constexpr float y = 1.f / 448.f;
  const float q = __fmul_rn(a, y);
  return __fmaf_rn(__fmaf_rn(-448.f, q, a), y, q);
}

// quant_span of N spans at once (aligned; N = 1, 2 or 4), span i from column c0 + i * step:
// the N maxima of a half-warp are reduced together, each step halving how many a lane
// holds, so that one division pass serves all 2 N groups; the row kernels are bound by
// instructions where every span reduces and divides for itself.
template <int N>
__device__ __forceinline__ void quant_spans(const float2 (*y)[4], int c0, int step, int cols, int lane, uint8_t* codes,
                                            float* scale, int64_t ld_scale) {
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = max3(fabsf(y[i][0].x), fabsf(y[i][0].y), fabsf(y[i][1].x));
    a[i] = max3(a[i], fabsf(y[i][1].y), fabsf(y[i][2].x));
    a[i] = max3(a[i], fabsf(y[i][2].y), fabsf(y[i][3].x));
    a[i] = max_nan(a[i], fabsf(y[i][3].y));
  }
  // lane bits from 3 down choose the span that the lane goes on with
  int o = 8;
#pragma unroll
  for (int m = N; m > 1; m >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < m / 2; ++i) {
      const float give = up ? a[i] : a[i + m / 2], keep = up ? a[i + m / 2] : a[i];
      a[i] = max_nan(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
    }
  }
#pragma unroll
  for (; o; o >>= 1) a[0] = max_nan(a[0], __shfl_xor_sync(0xFFFFFFFFu, a[0], o));
  constexpr int kShift = N == 4 ? 2 : N == 2 ? 3 : 4;  // lanes of a group: its span is (lane & 15) >> kShift
  const int mine = c0 + ((lane & 15) >> kShift) * step + (lane >> 4) * 128;
  const bool store = (lane & ((1 << kShift) - 1)) == 0 && mine < cols;
  if (__all_sync(0xFFFFFFFFu, mine >= cols || (a[0] >= 7.8886091e-31f && a[0] <= 3.4028235e38f))) {
    const float r = __fdiv_rn(448.f, a[0]);
    if (store) scale[int64_t(mine >> 7) * ld_scale] = over_448(a[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 ri = dup(__shfl_sync(0xFFFFFFFFu, r, (lane & 16) | (i << kShift)));
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = uint32_t(__nv_cvt_float2_to_fp8x2(mul2(y[i][j], ri), __NV_SATFINITE, __NV_E4M3));
      const int c = c0 + i * step + 8 * lane;
      if (c < cols) *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  } else {  // a zero, tiny, infinite or NaN group among them
    const QScale q = qscale(__float_as_uint(a[0]), 448.f);
    if (store) scale[int64_t(mine >> 7) * ld_scale] = q.s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int from = (lane & 16) | (i << kShift);
      QScale qi;
      qi.s = __shfl_sync(0xFFFFFFFFu, q.s, from);
      qi.r = __shfl_sync(0xFFFFFFFFu, q.r, from);
      qi.mode = __shfl_sync(0xFFFFFFFFu, q.mode, from);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = y[i][j].x, v[2 * j + 1] = y[i][j].y;
      const int c = c0 + i * step + 8 * lane;
      if (c < cols) *reinterpret_cast<uint2*>(codes + c) = codes_e4m3(v, qi);
    }
  }
}

__device__ __forceinline__ void unpack8(const uint4& w, float2* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2* v) {
  return make_uint4(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y), pack2(v[2].x, v[2].y), pack2(v[3].x, v[3].y));
}

// bf16(a + b), each pair's sums rounded once
__device__ __forceinline__ uint4 add_bf16(const uint4& a, const uint4& b) {
  auto add = [](uint32_t x, uint32_t y) {
    const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&s);
  };
  return make_uint4(add(a.x, b.x), add(a.y, b.y), add(a.z, b.z), add(a.w, b.w));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

__device__ __forceinline__ int64_t load_id(const void* ids, int bits, int64_t i) {
  return bits == 64 ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// ---------------------------------------------------------------- embedding lookup

constexpr int kRowWarps = 8;
constexpr int kSpans = 4;                // spans of a row that one warp copies
constexpr int kSeg = kSpans * kSpan;     // their columns

// 8192 tokens of a bf16 128256 x 4096 table: 17.2 us for 134 MB, 7.8 TB/s (a copy: 6.8; the
// rows of tokens that occur again come from L2)
template <bool VEC, bool FP8>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_embed(const void* __restrict__ table, const float* __restrict__ tscale, int64_t rows, int cols, int64_t ldt,
            const void* __restrict__ ids, int id_bits, int64_t n, float scale, __nv_bfloat16* __restrict__ out,
            int64_t ldo, int segs) {
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / segs;
  if (t >= n) return;
  const int c0 = int(item - t * segs) * kSeg;
  const int64_t id = load_id(ids, id_bits, t);
  const bool seen = id >= 0 && id < rows;
  float v[kSpans][8] = {};
  if (seen) {
    if (FP8) {
      const uint8_t* row = static_cast<const uint8_t*>(table) + id * ldt;
      const float* srow = tscale + (id >> 7) * ((cols + 127) >> 7);
      uint2 q[kSpans];
      float qs[kSpans];
#pragma unroll
      for (int j = 0; j < kSpans; ++j) {
        const int c = c0 + kSpan * j + 8 * lane;
        if (VEC && c < cols) q[j] = __ldg(reinterpret_cast<const uint2*>(row + c)), qs[j] = __ldg(srow + (c >> 7));
      }
#pragma unroll
      for (int j = 0; j < kSpans; ++j) {
        if (VEC) {
          const int c = c0 + kSpan * j + 8 * lane;
          if (c >= cols) continue;
          decode8(q[j], v[j]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = __fmul_rn(v[j][e], qs[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = c0 + kSpan * j + 32 * e + lane;
            if (c < cols) v[j][e] = __fmul_rn(decode1(row[c]), __ldg(srow + (c >> 7)));
          }
        }
      }
    } else {
      const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(table) + id * ldt;
#pragma unroll
      for (int j = 0; j < kSpans; ++j) load_bf16<VEC>(row, c0 + kSpan * j, cols, lane, v[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kSpans; ++j) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = seen ? __fmul_rn(v[j][e], scale) : 0.f;
    store_bf16<VEC>(out + t * ldo, c0 + kSpan * j, cols, lane, v[j]);
  }
}

// ---------------------------------------------------------------- tokens sorted by id
// By (id, position), so that equal ids keep their order.  Ids outside [0, rows) become
// `rows` (last).  The same launch writes the gradient's rows as zeros (ZeroRows), which
// most of a large table stays.

constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = 32;
// Zeros of a CTA, in address order: 16 KB (1.05 GB at 7.6 TB/s, 6.4 at 1 MB a CTA); beside
// the radix sort, whose clusters of large CTAs are slow to launch, an eighth of an SM's
// share (1.05 GB: 354 us at 32 KB, 210 at 128 KB, 177 at 512 KB).
constexpr int kZeroMin = 16384, kZeroRows = 8192;

struct ZeroRows {
  unsigned char* out;
  int64_t rows, pitch;     // bytes
  int row_bytes, each;     // rows a CTA
  int word;                // bytes a store: 16, 4 or 2
};

// CTA `cta` of the zeros
__device__ __forceinline__ void write_zeros(const ZeroRows& z, int64_t cta) {
  const int64_t v0 = cta * z.each;
  if (v0 >= z.rows) return;
  const int count = int(min(int64_t(z.each), z.rows - v0)), per = z.row_bytes / z.word;
  for (int i = threadIdx.x; i < count * per; i += blockDim.x) {
    const int r = i / per;
    unsigned char* o = z.out + (v0 + r) * z.pitch + int64_t(i - r * per) * z.word;
    if (z.word == 16)
      *reinterpret_cast<uint4*>(o) = make_uint4(0u, 0u, 0u, 0u);
    else if (z.word == 4)
      *reinterpret_cast<uint32_t*>(o) = 0u;
    else
      *reinterpret_cast<uint16_t*>(o) = 0;
  }
}

__device__ __forceinline__ uint32_t sort_key(const void* ids, int bits, int64_t i, int rows) {
  const int64_t id = load_id(ids, bits, i);
  return id >= 0 && id < rows ? uint32_t(id) : uint32_t(rows);
}

// Up to 8192 tokens, first half: each CTA sorts a chunk of 256 tokens by a bitonic network
// over distinct (id, position) keys, in registers and shared memory.  key, pos: the
// chunks one after another, padded to whole chunks with maximal ids.
constexpr int kChunk = 32 * kRowWarps, kChunkTokens = 8192;

__global__ void __launch_bounds__(kChunk)
    k_embed_chunks(const void* __restrict__ ids, int id_bits, int n, int rows, uint32_t* __restrict__ key,
                   uint32_t* __restrict__ pos, const ZeroRows z) {
  __shared__ uint64_t swap[2][kChunk];
  const int tid = threadIdx.x;
  after_previous();
  next_may_start();
  const int chunks = (n + kChunk - 1) / kChunk;
  if (int(blockIdx.x) >= chunks) {
    write_zeros(z, int(blockIdx.x) - chunks);
    return;
  }
  const int i = int(blockIdx.x) * kChunk + tid;
  uint64_t v = ~uint64_t(0);
  if (i < n) v = (uint64_t(sort_key(ids, id_bits, i, rows)) << 32) | uint32_t(i);
  int flip = 0;
  for (int k = 2; k <= kChunk; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      uint64_t o;
      if (j >= 32) {
        swap[flip][tid] = v;
        __syncthreads();
        o = swap[flip][tid ^ j];
        flip ^= 1;
      } else {
        o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
      }
      const bool low = ((tid & j) == 0) == ((tid & k) == 0);  // keeps the smaller of the two
      v = (v < o) == low ? v : o;
    }
  key[i] = uint32_t(v >> 32);
  pos[i] = uint32_t(v);
}

// Second half: a token's place is its place in its chunk and, by a binary search in each
// other chunk, the number of tokens there before it: ids up to its own in the chunks
// before, smaller ids in the chunks after.  Four threads a token share the chunks.
// A radix sort on a cluster (below) takes as long for 8192 tokens, but its large CTAs hold
// up the zeros beside it (8192 tokens of a 128256 x 4096 table: 169 us in all, 182 with it);
// comparing every token with every other in one launch took 20 us more.
constexpr int kPlaceEach = 64;
__global__ void __launch_bounds__(4 * kPlaceEach)
    k_embed_place(const uint32_t* __restrict__ key, const uint32_t* __restrict__ pos, int n, uint2* __restrict__ out) {
  __shared__ __align__(16) uint32_t all[kChunkTokens];
  const int tid = threadIdx.x, chunks = (n + kChunk - 1) / kChunk;
  after_previous();
  next_may_start();
#pragma unroll 8
  for (int i = tid; i < chunks * (kChunk / 4); i += 4 * kPlaceEach)
    reinterpret_cast<uint4*>(all)[i] = reinterpret_cast<const uint4*>(key)[i];
  const int i = int(blockIdx.x) * kPlaceEach + (tid >> 2);
  const uint32_t p = i < chunks * kChunk ? pos[i] : 0u;
  __syncthreads();
  const int home = i / kChunk;
  const uint32_t mine = home < chunks ? all[i] : 0xFFFFFFFFu;
  int place = 0;
  for (int c = tid & 3; c < chunks; c += 4) {
    if (c == home) {
      place += i - home * kChunk;
      continue;
    }
    const uint32_t* k = all + c * kChunk;
    const uint32_t first = c < home ? mine + 1 : mine;  // the smallest id that does not come before it
    int at = 0;
#pragma unroll
    for (int step = kChunk / 2; step; step >>= 1)
      if (k[at + step - 1] < first) at += step;
    place += at + (k[at] < first ? 1 : 0);
  }
  place += __shfl_xor_sync(0xFFFFFFFFu, place, 1);
  place += __shfl_xor_sync(0xFFFFFFFFu, place, 2);
  if ((tid & 3) == 0 && mine != 0xFFFFFFFFu) out[place] = make_uint2(mine, p);  // (not the padding)
}

// More tokens: a stable least-significant-digit radix sort on a cluster of eight CTAs (the
// grid's first), each owning a contiguous eighth of the tokens.  Per digit: CTA histograms,
// exchanged through distributed shared memory and scanned by every CTA; then ranks in
// token order, 1024 x kSortKeys tokens a round, by warp match and per-warp counters; the pairs
// go to the other buffer, which the cluster barrier makes visible.
constexpr int kDigit = 9, kBins = 1 << kDigit, kSortKeys = 4;

struct SortSmem {
  uint32_t hist[kBins];               // this CTA's count of every digit (read by the whole cluster)
  uint32_t base[kBins];               // where this CTA's next token of a digit goes
  uint32_t half[2][kBins];            // a round's count of every digit in warps 0-15, 16-31
  uint32_t warp_sum[kSortWarps];
  uint16_t count[kSortWarps][kBins];  // a round's counts, then offsets, by warp
};

__global__ void __launch_bounds__(kSortThreads, 1) __cluster_dims__(kSortCtas, 1, 1)
    k_embed_sort(const void* __restrict__ ids, int id_bits, int n, int rows, int passes, uint2* __restrict__ buf0,
                 uint2* __restrict__ buf1, const ZeroRows z) {
  __shared__ SortSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = int(cluster_rank());
  const int seg = (n + kSortCtas - 1) / kSortCtas;
  const int lo = min(n, rank * seg), hi = min(n, lo + seg);
  after_previous();
  next_may_start();
  if (blockIdx.x >= kSortCtas) {
    write_zeros(z, blockIdx.x - kSortCtas);
    return;
  }
  for (int p = 0; p < passes; ++p) {
    const uint2* src = (p & 1) ? buf1 : buf0;  // pass 0 reads the ids themselves
    uint2* dst = (p & 1) ? buf0 : buf1;
    const int shift = p * kDigit;
    auto key_at = [&](int i) -> uint2 {
      return p > 0 ? __ldcg(src + i) : make_uint2(sort_key(ids, id_bits, i, rows), uint32_t(i));
    };
    if (tid < kBins) sm.hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kSortThreads) atomicAdd(&sm.hist[(key_at(i).x >> shift) & (kBins - 1)], 1u);
    cluster_sync();
    // exclusive scan over (digit, CTA): thread d < kBins holds digit d
    uint32_t before = 0, total = 0;
    if (tid < kBins) {
      const uint32_t at = smem_addr(&sm.hist[tid]);
      uint32_t h[kSortCtas];
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(h[c]) : "r"(map_rank(at, uint32_t(c))) : "memory");
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        if (c < rank) before += h[c];
        total += h[c];
      }
    }
    uint32_t x = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm.warp_sum[warp] = x;
    __syncthreads();
    if (tid < kBins) {
      uint32_t prior = lane < warp ? sm.warp_sum[lane] : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) prior += __shfl_xor_sync(0xFFFFFFFFu, prior, o);
      sm.base[tid] = prior + x - total + before;
    }
    // ranks, in token order
    for (int r0 = lo; r0 < hi; r0 += kSortThreads * kSortKeys) {
      uint4* clear = reinterpret_cast<uint4*>(sm.count);
      for (int i = tid; i < kSortWarps * kBins / 8; i += kSortThreads) clear[i] = make_uint4(0u, 0u, 0u, 0u);
      uint2 kv[kSortKeys];
      uint32_t off[kSortKeys];
      const int w0 = r0 + warp * 32 * kSortKeys;
#pragma unroll
      for (int j = 0; j < kSortKeys; ++j) {
        const int i = w0 + 32 * j + lane;
        if (i < hi) kv[j] = key_at(i);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSortKeys; ++j) {
        const bool on = w0 + 32 * j + lane < hi;
        const uint32_t d = on ? (kv[j].x >> shift) & (kBins - 1) : kBins;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t below = __popc(peers & ((1u << lane) - 1u));
        uint32_t prior = 0;
        if (on) prior = sm.count[warp][d];
        __syncwarp();
        if (on && below == 0) sm.count[warp][d] = uint16_t(prior + __popc(peers));
        __syncwarp();
        off[j] = prior + below;
      }
      __syncthreads();
      {  // counts -> offsets of each warp within its half of the warps
        const int d = tid & (kBins - 1), h = tid >> kDigit;
        uint32_t c[kSortWarps / 2], run = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps / 2; ++w) c[w] = sm.count[h * (kSortWarps / 2) + w][d];
#pragma unroll
        for (int w = 0; w < kSortWarps / 2; ++w) {
          sm.count[h * (kSortWarps / 2) + w][d] = uint16_t(run);
          run += c[w];
        }
        sm.half[h][d] = run;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSortKeys; ++j) {
        if (w0 + 32 * j + lane >= hi) continue;
        const uint32_t d = (kv[j].x >> shift) & (kBins - 1);
        dst[sm.base[d] + (warp >= kSortWarps / 2 ? sm.half[0][d] : 0u) + sm.count[warp][d] + off[j]] = kv[j];
      }
      __syncthreads();
      if (tid < kBins) sm.base[tid] += sm.half[0][tid] + sm.half[1][tid];
    }
    __threadfence();
    cluster_sync();  // the next pass reads other CTAs' pairs; their histograms are done being read
  }
}

// ---------------------------------------------------------------- embedding gradient

// dT[v] (+)= f * sum of dY[t] over the tokens t of id v, summed in fp32 in token
// order.  The sorted tokens are cut into pieces.  A run of equal ids inside
// one piece is summed and its row written by the piece's CTA; of a run that crosses a
// piece's end each piece's part is summed first, so that a token that fills the batch
// is shared out over the whole GPU, and k_embed_join adds the parts in order.  No
// atomics: the same batch gives the same bits.
// Slot of a piece's part: 2c for the one that starts with piece c, 2c + 1 otherwise.
// A piece is 32 tokens, or 16 up to 2048 tokens, where its rounds of loads are what
// takes the time (300 tokens: 14.1 us with 32, 11.6 with 16; 8192: 31.6 and 36.6).
constexpr int kMaxPiece = 32, kBatch = 8;   // tokens of a piece at most; rows of dY in flight
constexpr int piece_of(int64_t n) { return n <= 2048 ? 16 : 32; }

template <bool VEC, typename Out>
__device__ __forceinline__ void write_sum(Out* row, int c0, int cols, int lane, float scale, int accumulate, float* acc) {
  if (accumulate) {
    float old[8];
    load_row<VEC>(row, c0, cols, lane, old);
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = fmaf(scale, acc[x], old[x]);
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = __fmul_rn(scale, acc[x]);
  }
  store_row<VEC>(row, c0, cols, lane, acc);
}

struct EmbedRows {
  const uint2* sorted;
  const __nv_bfloat16* dy;
  float* sums;            // [2 pieces][ldp]
  int64_t ld, rows, ldo;
  int n, cols, ldp, accumulate, piece;
  int groups;             // CTAs of a piece: kRowWarps spans each
  float scale;
};

// In all 8192 tokens of a 128256 x 4096 bf16 table take 169 us: 1.05 GB of zeros and sums
// written and 67 MB read, 6.6 TB/s.
template <bool VEC, typename Out>
__global__ void __launch_bounds__(32 * kRowWarps, 4) k_embed_rows(const EmbedRows a, Out* __restrict__ out) {
  __shared__ uint32_t key[kMaxPiece + 2], pos[kMaxPiece];  // key[1 + i]: token i of the piece; 0, len + 1: its neighbours
  const int tid = threadIdx.x, lane = tid & 31;
  after_previous();
  next_may_start();
  const int piece = int(blockIdx.x) / a.groups;
  const int b = piece * a.piece, len = min(a.piece, a.n - b);
  if (tid < len + 2) {
    const int i = b + tid - 1;
    const uint2 kv = i >= 0 && i < a.n ? a.sorted[i] : make_uint2(0xFFFFFFFFu, 0u);
    key[tid] = kv.x;
    if (tid >= 1 && tid <= len) pos[tid - 1] = kv.y;
  }
  __syncthreads();
  const int c0 = ((int(blockIdx.x) - piece * a.groups) * kRowWarps + (tid >> 5)) * kSpan;
  if (c0 >= a.cols) return;
  float acc[8] = {};
  int start = 0;  // first token of the run being summed
  for (int i0 = 0; i0 < len; i0 += kBatch) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < len) w[k] = load_packed<VEC>(a.dy + int64_t(pos[i0 + k]) * a.ld, c0, a.cols, lane);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k;
      if (i >= len) continue;
      float v[8];
      unpack8(w[k], v);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[x]);
      const uint32_t id = key[1 + i];
      if (i + 1 < len && key[2 + i] == id) continue;
      // the run (or this piece's part of it) ends here
      if (id < uint32_t(a.rows)) {
        const bool whole = (start > 0 || key[0] != id) && (i + 1 < len || key[len + 1] != id);
        if (whole)
          write_sum<VEC>(out + int64_t(id) * a.ldo, c0, a.cols, lane, a.scale, a.accumulate, acc);
        else  // (a slot's values lie as the lanes hold them: VEC or not, its reader holds the same)
          store_f32<true>(a.sums + int64_t(2 * piece + (start > 0 ? 1 : 0)) * a.ldp, c0, a.ldp, lane, acc);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = 0.f;
      start = i + 1;
    }
  }
}

// Up to kFewTokens tokens: the whole gradient in one launch, without a sort.  The CTAs of
// token t (one a group of spans) look through all ids: if t is the first of its id they
// sum that id's tokens in order.  The others write zeros into the rows that no token names.
constexpr int kFewTokens = 256;
template <bool VEC, typename Out>
__global__ void __launch_bounds__(32 * kRowWarps, 4)
    k_embed_few(const EmbedRows a, const void* __restrict__ ids, int id_bits, const ZeroRows z, Out* __restrict__ out) {
  __shared__ uint32_t list[kFewTokens], named[kZeroRows / 32];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31;
  after_previous();
  next_may_start();
  const uint32_t id = tid < a.n ? sort_key(ids, id_bits, tid, int(a.rows)) : uint32_t(a.rows);
  if (int(blockIdx.x) >= a.n * a.groups) {
    const int64_t cta = int64_t(blockIdx.x) - int64_t(a.n) * a.groups, v0 = cta * z.each;
    for (int i = tid; i < (z.each + 31) / 32; i += 32 * kRowWarps) named[i] = 0;
    __syncthreads();
    const int64_t at = int64_t(id) - v0;
    const bool mine = id < uint32_t(a.rows) && at >= 0 && at < z.each;
    if (mine) atomicOr(&named[at >> 5], 1u << (at & 31));
    if (!__syncthreads_or(mine)) {
      write_zeros(z, cta);
      return;
    }
    const int rows = int(min(int64_t(z.each), z.rows - v0));
    for (int r = tid >> 5; r < rows; r += kRowWarps) {
      if ((named[r >> 5] >> (r & 31)) & 1u) continue;
      unsigned char* o = z.out + (v0 + r) * z.pitch;
      for (int i = lane * z.word; i < z.row_bytes; i += 32 * z.word) {
        if (z.word == 16)
          *reinterpret_cast<uint4*>(o + i) = make_uint4(0u, 0u, 0u, 0u);
        else if (z.word == 4)
          *reinterpret_cast<uint32_t*>(o + i) = 0u;
        else
          *reinterpret_cast<uint16_t*>(o + i) = 0;
      }
    }
    return;
  }
  const int t = int(blockIdx.x) / a.groups;
  list[tid] = id;
  __syncthreads();
  const uint32_t want = list[t];
  if (want >= uint32_t(a.rows)) return;
  const bool same = id == want;
  if (__syncthreads_or(same && tid < t)) return;  // (also: every thread has read list[t])
  if (tid < 32) {  // its tokens, in order
    int n = 0;
    for (int i0 = 0; i0 < kFewTokens; i0 += 32) {
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, list[i0 + lane] == want);
      __syncwarp();
      if ((hit >> lane) & 1u) list[n + __popc(hit & ((1u << lane) - 1u))] = uint32_t(i0 + lane);
      n += __popc(hit);
      __syncwarp();
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int c0 = ((int(blockIdx.x) - t * a.groups) * kRowWarps + (tid >> 5)) * kSpan;
  if (c0 >= a.cols) return;
  float acc[8] = {};
  for (int i0 = 0; i0 < count; i0 += kBatch) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < count) w[k] = load_packed<VEC>(a.dy + int64_t(list[i0 + k]) * a.ld, c0, a.cols, lane);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k >= count) continue;
      float v[8];
      unpack8(w[k], v);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[x]);
    }
  }
  write_sum<VEC>(out + int64_t(want) * a.ldo, c0, a.cols, lane, a.scale, a.accumulate, acc);
}

// rows whose run begins in piece blockIdx.x / groups and goes on past its end
template <bool VEC, typename Out>
__global__ void __launch_bounds__(32 * kRowWarps) k_embed_join(const EmbedRows a, Out* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int piece = int(blockIdx.x) / a.groups, b = piece * a.piece, e = b + a.piece;
  after_previous();
  next_may_start();
  if (e >= a.n) return;
  const uint32_t id = a.sorted[e - 1].x, after = a.sorted[e].x, first = a.sorted[b].x;
  const uint32_t before = a.sorted[max(b, 1) - 1].x;
  const bool from_start = first == id;
  if (after != id || id >= uint32_t(a.rows) || (from_start && b > 0 && before == id)) return;  // (began in an earlier piece)
  const int c0 = ((int(blockIdx.x) - piece * a.groups) * kRowWarps + int(threadIdx.x >> 5)) * kSpan;
  if (c0 >= a.cols) return;
  float acc[8];
  load_f32<true>(a.sums + int64_t(2 * piece + (from_start ? 0 : 1)) * a.ldp, c0, a.ldp, lane, acc);
  // the pieces after it that start with the same id, 32 at a time
  for (int p = piece + 1;; p += 32) {
    const int at = (p + lane) * a.piece;
    const uint32_t same = __ballot_sync(0xFFFFFFFFu, at < a.n && a.sorted[at].x == id);
    const int count = same == 0xFFFFFFFFu ? 32 : __ffs(int(~same)) - 1;
    for (int k0 = 0; k0 < count; k0 += 8) {
      float v[8][8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < count) load_f32<true>(a.sums + int64_t(2 * (p + k0 + k)) * a.ldp, c0, a.ldp, lane, v[k]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < count) {
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[k][x]);
        }
    }
    if (count < 32) break;
  }
  write_sum<VEC>(out + int64_t(id) * a.ldo, c0, a.cols, lane, a.scale, a.accumulate, acc);
}

// ---------------------------------------------------------------- norm

// One CTA per row: warp w holds spans w, w + warps, ... of it in registers.
struct NormArgs {
  const __nv_bfloat16 *x, *res, *w;
  __nv_bfloat16 *h, *y;
  uint8_t* codes;
  float *scale, *rstd;
  int64_t ldx, ldr, ldh, ldy, ldc, lds;
  float eps;
  int cols;
};

constexpr int row_threads(int vpt) { return vpt <= 4 ? 512 : 1024; }

template <bool VEC, int VPT>
__global__ void __launch_bounds__(row_threads(VPT)) k_norm(const NormArgs a) {
  after_previous();
  next_may_start();
  __shared__ float part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t t = blockIdx.x;
  float h[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) load_bf16<VEC>(a.x + t * a.ldx, (warp + i * warps) * kSpan, a.cols, lane, h[i]);
  if (a.res) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c0 = (warp + i * warps) * kSpan;
      float r[8];
      load_bf16<VEC>(a.res + t * a.ldr, c0, a.cols, lane, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __nv_bfloat16 b = __hadd(__float2bfloat16_rn(h[i][e]), __float2bfloat16_rn(r[e]));  // (both exact)
        h[i][e] = __bfloat162float(b);
      }
      if (a.h) store_bf16<VEC>(a.h + t * a.ldh, c0, a.cols, lane, h[i]);
    }
  }
  float2 s2 = dup(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 v = make_float2(h[i][e], h[i][e + 1]);
      s2 = fma2(v, v, s2);
    }
  float ss = warp_sum(s2.x + s2.y);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = warp_sum(lane < warps ? part[lane] : 0.f);
  const float rstd = rsqrtf(__fadd_rn(__fdiv_rn(ss, float(a.cols)), a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c0 = (warp + i * warps) * kSpan;
    if (c0 >= a.cols) break;
    float w[8];
    load_bf16<VEC>(a.w, c0, a.cols, lane, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = __fmul_rn(__fmul_rn(h[i][e], rstd), w[e]);
    if (a.y) store_bf16<VEC>(a.y + t * a.ldy, c0, a.cols, lane, h[i]);
    if (a.codes) quant_span<VEC>(h[i], c0, a.cols, lane, a.codes + t * a.ldc, a.scale + t, a.lds);
  }
}

// 16 bytes into shared memory without a register (zeros where !on)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread's copies have landed
__device__ __forceinline__ void copy_wait(int n) {
  switch (n) {
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}

// Many rows: resident CTAs walk the rows blockIdx.x, + gridDim.x, ..., each thread
// copying its own vectors of the next `depth` - 1 rows into a ring in shared memory, so
// that loads are in flight while a row waits for its sum (with a CTA per row they are
// not).  A thread reads only what it copied: no barrier but the sum's.  8192 rows of 4096
// with a residual: 40.6 us, 5.8 TB/s of the 7 bytes a value (a copy: 6.8), where one CTA a
// row takes 50 (issue slots are busy half of the time).
template <int VPT>
__global__ void __launch_bounds__(VPT <= 2 ? 1024 : 512, 1) k_norm_many(const NormArgs a, int64_t n, int depth) {
  after_previous();
  next_may_start();
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float part[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int ins = a.res ? 2 : 1;
  const uint32_t step = blockDim.x * 16u;                    // one vector of every thread
  const uint32_t row_bytes = uint32_t(ins) * VPT * step;     // a slot of the ring
  const uint32_t mine = smem_addr(ring) + threadIdx.x * 16u;
  uint4 w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) w[i] = load_packed<true>(a.w, (warp + i * warps) * kSpan, a.cols, lane);
  auto fetch = [&](int64_t t, int slot) {
    if (t < n) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (warp + i * warps) * kSpan + 8 * lane;
        const bool on = c < a.cols;
        const uint32_t at = mine + uint32_t(slot) * row_bytes + uint32_t(i) * step;
        copy16(at, a.x + t * a.ldx + (on ? c : 0), on);
        if (a.res) copy16(at + VPT * step, a.res + t * a.ldr + (on ? c : 0), on);
      }
    }
    copy_commit();
  };
  int64_t next = blockIdx.x;
  for (int s = 0; s + 1 < depth; ++s, next += gridDim.x) fetch(next, s);
  int slot = 0, flip = 0;
  for (int64_t t = blockIdx.x; t < n; t += gridDim.x, next += gridDim.x, flip ^= 1) {
    fetch(next, slot == 0 ? depth - 1 : slot - 1);  // the slot read last
    copy_wait(depth - 1);
    float2 h[VPT][4];
    float2 s2 = dup(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t at = mine + uint32_t(slot) * row_bytes + uint32_t(i) * step;
      uint4 b = shared16(at);
      if (a.res) {
        b = add_bf16(b, shared16(at + VPT * step));
        const int c = (warp + i * warps) * kSpan + 8 * lane;
        if (c < a.cols) *reinterpret_cast<uint4*>(a.h + t * a.ldh + c) = b;
      }
      unpack8(b, h[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(h[i][e], h[i][e], s2);
    }
    slot = slot + 1 == depth ? 0 : slot + 1;
    float ss = warp_sum(s2.x + s2.y);
    if (lane == 0) part[flip][warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < warps ? part[flip][lane] : 0.f);
    const float rstd = rsqrtf(__fadd_rn(__fdiv_rn(ss, float(a.cols)), a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float2 g[4];
      unpack8(w[i], g);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[i][e] = mul2(mul2(h[i][e], dup(rstd)), g[e]);
      const int c = (warp + i * warps) * kSpan + 8 * lane;
      if (a.y && c < a.cols) *reinterpret_cast<uint4*>(a.y + t * a.ldy + c) = pack8(h[i]);
    }
    if (a.codes)
      quant_spans<VPT>(h, warp * kSpan, warps * kSpan, a.cols, lane, a.codes + t * a.ldc, a.scale + t, a.lds);
  }
}

// a warp quantises N spans of a row.  IN: x's rows are whole vectors; OUT: the codes' are.
template <bool IN, bool OUT, int N>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_quant_rows(const __nv_bfloat16* __restrict__ x, int64_t ldx, int64_t n, int cols, uint8_t* __restrict__ codes,
                 int64_t ldc, float* __restrict__ scale, int64_t lds, int segs) {
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / segs;
  if (t >= n) return;
  const int c0 = int(item - t * segs) * N * kSpan;
  if (OUT) {
    uint4 w[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
      w[j] = IN ? load_packed<true>(x + t * ldx, c0 + kSpan * j, cols, lane)
                : load_shifted(x + t * ldx, c0 + kSpan * j, cols, lane);
    float2 v[N][4];
#pragma unroll
    for (int j = 0; j < N; ++j) unpack8(w[j], v[j]);
    quant_spans<N>(v, c0, kSpan, cols, lane, codes + t * ldc, scale + t, lds);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (c0 + kSpan * j >= cols) break;
      float v[8];
      load_bf16<false>(x + t * ldx, c0 + kSpan * j, cols, lane, v);
      quant_span<false>(v, c0 + kSpan * j, cols, lane, codes + t * ldc, scale + t, lds);
    }
  }
}

// The weight gradient's operands in bf16 at pitches of their own: scale * code of E4M3
// rows with one scale per 128 values (cols is a multiple of 16, so every vector is
// aligned), by the first x_items warps; and, by the others, dY where its own pitch does
// not serve.
struct DwInputs {
  const uint8_t* codes;
  const float* scale;
  const __nv_bfloat16* dy;
  __nv_bfloat16 *x_out, *dy_out;
  int64_t ldc, lds, ldo, ldy, ldyo, x_items, items;
  int cols, x_spans, rows, y_spans;
};

__global__ void __launch_bounds__(32 * kRowWarps) k_dw_inputs(const DwInputs a) {
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item < a.x_items) {
    const int64_t t = item / a.x_spans;
    const int c = int(item - t * a.x_spans) * kSpan + 8 * lane;
    if (c >= a.cols) return;
    float v[8];
    decode8(__ldg(reinterpret_cast<const uint2*>(a.codes + t * a.ldc + c)), v);
    const float s = __ldg(a.scale + int64_t(c >> 7) * a.lds + t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], s);
    *reinterpret_cast<uint4*>(a.x_out + t * a.ldo + c) = pack8(v);
  } else if (item < a.items) {
    const int64_t i = item - a.x_items, t = i / a.y_spans;
    const int c0 = int(i - t * a.y_spans) * kSpan, c = c0 + 8 * lane;
    const uint4 w = load_shifted(a.dy + t * a.ldy, c0, a.rows, lane);
    if (c < a.rows) *reinterpret_cast<uint4*>(a.dy_out + t * a.ldyo + c) = w;  // (the pitch covers whole vectors)
  }
}

// dw (+)= sum over few tokens of dy[t]^T bf16(x[t]): a CTA holds its 64 rows of dY^T and 256
// columns of X in shared memory, 16 tokens at a time, and writes a 64 x 256 tile, a thread 8
// rows x 8 columns of it.  Bound by the write for a token or two (4096 x 4096: 8.4 us, 4 TB/s), by
// fp32 multiply-adds then; one launch, where the products on the tensor cores convert X first.
constexpr int kFewRows = 64, kFewCols = 256, kFewDeep = 16;  // (tokens in shared memory at once)
__global__ void __launch_bounds__(256)
    k_dw_few(const __nv_bfloat16* __restrict__ dy, int64_t ldy, const uint8_t* __restrict__ codes, int64_t ldc,
             const float* __restrict__ scale, int64_t lds, int n, int rows, int cols, __nv_bfloat16* __restrict__ dw,
             int64_t ldw, int accumulate) {
  __shared__ __align__(16) float x[kFewDeep][kFewCols], y[kFewDeep][kFewRows];
  const int tid = threadIdx.x;
  const int col_tiles = (cols + kFewCols - 1) / kFewCols;
  const int r0 = int(blockIdx.x) / col_tiles * kFewRows, c0 = int(blockIdx.x) % col_tiles * kFewCols;
  after_previous();
  next_may_start();
  const int lane = tid & 31, r1 = 8 * (tid >> 5), c1 = 8 * lane;
  float2 acc[8][4] = {};
  for (int t0 = 0; t0 < n; t0 += kFewDeep) {
    const int deep = min(kFewDeep, n - t0);
    if (t0) __syncthreads();
    for (int i = tid; i < deep * (kFewCols / 8); i += 256) {  // (cols is a multiple of 16)
      const int t = i / (kFewCols / 8), c = 8 * (i % (kFewCols / 8));
      float v[8] = {};
      if (c0 + c < cols) {
        decode8(__ldg(reinterpret_cast<const uint2*>(codes + (t0 + t) * ldc + c0 + c)), v);
        const float s = __ldg(scale + int64_t((c0 + c) >> 7) * lds + t0 + t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __bfloat162float(__float2bfloat16_rn(__fmul_rn(v[e], s)));
      }
      *reinterpret_cast<float4*>(&x[t][c]) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(&x[t][c + 4]) = make_float4(v[4], v[5], v[6], v[7]);
    }
    for (int i = tid; i < deep * kFewRows; i += 256) {
      const int t = i / kFewRows, r = i % kFewRows;
      y[t][r] = r0 + r < rows ? __bfloat162float(dy[(t0 + t) * ldy + r0 + r]) : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < deep; ++t) {
      const float4 a = *reinterpret_cast<const float4*>(&x[t][c1]), b = *reinterpret_cast<const float4*>(&x[t][c1 + 4]);
      const float2 xv[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float2 f = dup(y[t][r1 + r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = fma2(f, xv[e], acc[r][e]);
      }
    }
  }
  if (c0 + c1 >= cols) return;
  const bool vec = ldw % 8 == 0 && (reinterpret_cast<uintptr_t>(dw) & 15) == 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = r0 + r1 + r;
    if (row >= rows) break;
    __nv_bfloat16* o = dw + int64_t(row) * ldw + c0 + c1;
    if (vec) {
      if (accumulate) {
        float2 old[4];
        unpack8(*reinterpret_cast<const uint4*>(o), old);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = make_float2(acc[r][e].x + old[e].x, acc[r][e].y + old[e].y);
      }
      *reinterpret_cast<uint4*>(o) = pack8(acc[r]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = e & 1 ? acc[r][e >> 1].y : acc[r][e >> 1].x;
        if (accumulate) v += __bfloat162float(o[e]);
        o[e] = __float2bfloat16_rn(v);
      }
    }
  }
}

// ---------------------------------------------------------------- norm gradient

struct NormGradArgs {
  const __nv_bfloat16 *dy, *h, *w, *dh;
  const float* rstd;
  __nv_bfloat16* dx;
  float* part;  // [gridDim.x][ldp] sums of dw over this CTA's rows
  int64_t ld_dy, ld_h, ld_dh, ld_dx, n;
  int cols, ldp;
};

// u = h rstd, t = dy w: dx = rstd (t - u mean(t u)) + dh, dw = sum over rows of dy u.
// CTAs walk the rows blockIdx.x, + gridDim.x, ...; a thread keeps its columns' dw.
template <bool VEC, int VPT>
__global__ void __launch_bounds__(1024, 1) k_norm_grad(const NormGradArgs a) {
  after_previous();
  next_may_start();
  __shared__ float part[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float dw[VPT][8] = {};
  int flip = 0;
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x, flip ^= 1) {
    const float rstd = a.rstd[t];
    float dy[VPT][8], u[VPT][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c0 = (warp + i * warps) * kSpan;
      float w[8];
      load_bf16<VEC>(a.dy + t * a.ld_dy, c0, a.cols, lane, dy[i]);
      load_bf16<VEC>(a.h + t * a.ld_h, c0, a.cols, lane, u[i]);
      load_bf16<VEC>(a.w, c0, a.cols, lane, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] *= rstd;
        dw[i][e] = fmaf(dy[i][e], u[i][e], dw[i][e]);
        dy[i][e] *= w[e];
        dot = fmaf(dy[i][e], u[i][e], dot);
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) part[flip][warp] = dot;
    __syncthreads();
    dot = warp_sum(lane < warps ? part[flip][lane] : 0.f) / float(a.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c0 = (warp + i * warps) * kSpan;
      float g[8] = {};
      if (a.dh) load_bf16<VEC>(a.dh + t * a.ld_dh, c0, a.cols, lane, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = fmaf(rstd, fmaf(-dot, u[i][e], dy[i][e]), g[e]);
      store_bf16<VEC>(a.dx + t * a.ld_dx, c0, a.cols, lane, g);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c0 = (warp + i * warps) * kSpan;
    if (c0 < a.cols) store_f32<VEC>(a.part + int64_t(blockIdx.x) * a.ldp, c0, a.cols, lane, dw[i]);
  }
}

// the same with the rows to come copied into a ring, as k_norm_many: 4099 rows of 8192 take
// 45.4 us with k_norm_dw, 5.9 TB/s of 8 bytes a value (67 without the ring)
template <int VPT>
__global__ void __launch_bounds__(1024, 1) k_norm_grad_many(const NormGradArgs a, int depth) {
  after_previous();
  next_may_start();
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float part[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int ins = a.dh ? 3 : 2;
  const uint32_t step = blockDim.x * 16u;
  const uint32_t row_bytes = uint32_t(ins) * VPT * step;
  const uint32_t mine = smem_addr(ring) + threadIdx.x * 16u;
  uint4 w[VPT];
  float2 dw[VPT][4] = {};
#pragma unroll
  for (int i = 0; i < VPT; ++i) w[i] = load_packed<true>(a.w, (warp + i * warps) * kSpan, a.cols, lane);
  auto fetch = [&](int64_t t, int slot) {
    if (t < a.n) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (warp + i * warps) * kSpan + 8 * lane;
        const bool on = c < a.cols;
        const uint32_t at = mine + uint32_t(slot) * row_bytes + uint32_t(i) * step;
        copy16(at, a.dy + t * a.ld_dy + (on ? c : 0), on);
        copy16(at + VPT * step, a.h + t * a.ld_h + (on ? c : 0), on);
        if (a.dh) copy16(at + 2 * VPT * step, a.dh + t * a.ld_dh + (on ? c : 0), on);
      }
    }
    copy_commit();
  };
  int64_t next = blockIdx.x;
  for (int s = 0; s + 1 < depth; ++s, next += gridDim.x) fetch(next, s);
  int slot = 0, flip = 0;
  float rnext = a.rstd[blockIdx.x];
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x, next += gridDim.x, flip ^= 1) {
    const float rstd = rnext;
    if (t + gridDim.x < a.n) rnext = a.rstd[t + gridDim.x];
    copy_wait(depth - 2);
    float2 dy[VPT][4], u[VPT][4];
    uint4 g[VPT];
    float2 d2 = dup(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t at = mine + uint32_t(slot) * row_bytes + uint32_t(i) * step;
      unpack8(shared16(at), dy[i]);
      unpack8(shared16(at + VPT * step), u[i]);
      g[i] = a.dh ? shared16(at + 2 * VPT * step) : make_uint4(0u, 0u, 0u, 0u);
      float2 f[4];
      unpack8(w[i], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[i][e] = mul2(u[i][e], dup(rstd));
        dw[i][e] = fma2(dy[i][e], u[i][e], dw[i][e]);
        dy[i][e] = mul2(dy[i][e], f[e]);
        d2 = fma2(dy[i][e], u[i][e], d2);
      }
    }
    fetch(next, slot == 0 ? depth - 1 : slot - 1);  // the slot read a row ago
    slot = slot + 1 == depth ? 0 : slot + 1;
    float dot = warp_sum(d2.x + d2.y);
    if (lane == 0) part[flip][warp] = dot;
    __syncthreads();
    dot = warp_sum(lane < warps ? part[flip][lane] : 0.f) / float(a.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (warp + i * warps) * kSpan + 8 * lane;
      float2 o[4];
      unpack8(g[i], o);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fma2(dup(rstd), fma2(dup(-dot), u[i][e], dy[i][e]), o[e]);
      if (c < a.cols) *reinterpret_cast<uint4*>(a.dx + t * a.ld_dx + c) = pack8(o);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c0 = (warp + i * warps) * kSpan;
    const float v[8] = {dw[i][0].x, dw[i][0].y, dw[i][1].x, dw[i][1].y, dw[i][2].x, dw[i][2].y, dw[i][3].x, dw[i][3].y};
    if (c0 < a.cols) store_f32<true>(a.part + int64_t(blockIdx.x) * a.ldp, c0, a.cols, lane, v);
  }
}

// dw = sum of the CTAs' parts in a fixed order: 32 columns a CTA, every 32nd part a warp
template <typename Out>
__global__ void __launch_bounds__(1024)
    k_norm_dw(const float* __restrict__ part, int parts, int ldp, int cols, int accumulate, Out* __restrict__ dw) {
  __shared__ float run[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  after_previous();
  next_may_start();
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) s += part[int64_t(p) * ldp + c];
  }
  run[warp][lane] = s;
  __syncthreads();
  s = warp_sum(run[lane][warp]);  // warp w: column w of the CTA's
  const int o = blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) {
    if (sizeof(Out) == 2) {
      __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(dw);
      if (accumulate) s += __bfloat162float(d[o]);
      d[o] = __float2bfloat16_rn(s);
    } else {
      float* d = reinterpret_cast<float*>(dw);
      if (accumulate) s += d[o];
      d[o] = s;
    }
  }
}

// ---------------------------------------------------------------- host

bool vec_ok(const void* p, int64_t ld, int values) { return aligned16(p) && ld % values == 0; }

// The norm's warps a row and spans a warp (VPT), within row_threads(VPT) threads for rows
// of up to 65536 columns.  Four spans a warp: what a warp does once a row is a third of
// its instructions with two (4096 columns: 43.5 us with two, 41.3 with four); also for 3 and
// 9 spans, although a quarter of the lanes idle (8192 rows and 700 rows: 8.6 and 3.9 us with
// four, 10.5 and 3.2 with two; 22.5 and 4.4, 23.9 and 4.6).  Two for 2, 5 and 6 spans, where
// few rows gain more than many lose (with two 8.7 and 2.8, 15.9 and 3.0, 17.7 and 3.1; with
// four 8.3 and 3.0, 15.6 and 3.8, 16.8 and 3.9).  One shape for any number of rows,
// so that a row's sum does not depend on the rows beside it.
// Rows that are not aligned are bound by their 2-byte accesses and want the warps (4095
// columns: 69 us with two spans, 94 us with four).
void norm_shape(int cols, bool vec, int* warps, int* vpt) {
  const int spans = (cols + kSpan - 1) / kSpan;
  *vpt = spans > 64 ? 8 : spans == 1 ? 1 : spans == 2 || spans == 5 || spans == 6 || (!vec && spans <= 32) ? 2 : 4;
  *warps = (spans + *vpt - 1) / *vpt;
}

int bits_of(int64_t x) {
  int b = 0;
  while (x) ++b, x >>= 1;
  return b;
}

struct EmbedGradPlan {
  size_t off_b0, off_b1, off_sums, bytes;
  int ldp, pieces;
};

EmbedGradPlan embed_grad_plan(int64_t n, int64_t cols) {
  EmbedGradPlan p;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.ldp = int((cols + kSpan - 1) / kSpan * kSpan);
  p.pieces = int((n + piece_of(n) - 1) / piece_of(n));
  p.off_b0 = 0;
  p.off_b1 = up(size_t(n) * 8);
  p.off_sums = p.off_b1 + up(size_t(n + kChunk) * 8);
  p.bytes = std::max<size_t>(256, p.off_sums + up(size_t(p.pieces) * 2 * size_t(p.ldp) * 4));
  return p;
}

// The ring of a kernel whose resident CTAs walk many rows: slots (0: it does not fit,
// or there are too few rows for it) and CTAs an SM, for `warps` warps a CTA and
// row_bytes of shared memory a row.  A CTA's barrier stalls it once a row, so an SM runs
// several of them, up to `most`, within `threads` threads (what the registers allow).
struct Ring {
  int depth, per_sm;
};

constexpr int kRingBytes = 224 * 1024, kMaxDepth = 8;

Ring ring_of(int warps, int row_bytes, int64_t n, int threads, int most) {
  Ring r;
  r.per_sm = std::max(1, std::min(most, threads / (32 * warps)));
  r.depth = std::min(kMaxDepth, (kRingBytes / r.per_sm - 1280) / row_bytes);
  if (r.depth < 3 || n < int64_t(2) * r.per_sm * sm_count()) r.depth = 0;
  return r;
}

struct NormGradPlan {
  int ctas, warps, vpt, depth, smem;
};

// vec: every row of the operands is 16-byte aligned and of whole vectors.  The direct
// kernel (depth 0) takes what the ring does not.
NormGradPlan norm_grad_plan(int64_t n, int cols, int ins, bool vec) {
  NormGradPlan p;
  const int spans = (cols + kSpan - 1) / kSpan;
  p.vpt = spans <= 32 ? 1 : spans <= 64 ? 2 : 8;
  p.warps = (spans + p.vpt - 1) / p.vpt;
  p.depth = 0, p.smem = 0;
  const int row = ins * p.vpt * p.warps * 512;
  const Ring r = ring_of(p.warps, row, n, 1024, 8);  // (each CTA leaves a part of dw)
  if (vec && p.vpt <= 2 && r.depth) p.depth = r.depth, p.smem = r.depth * row;
  // as few CTAs as give every one the same number of rows, or one less
  const int64_t most = int64_t(sm_count()) * r.per_sm, each = (n + most - 1) / most;
  p.ctas = n > 0 ? int((n + each - 1) / each) : 0;
  return p;
}

}  // namespace

int launch_embed(const EmbedArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = a.kind == BQ_ROWS_FP8;
  const bool vec = a.cols % 8 == 0 && vec_ok(a.out, a.ldo, 8) &&
                   (fp8 ? (reinterpret_cast<uintptr_t>(a.table) & 7) == 0 && a.ldt % 8 == 0 : vec_ok(a.table, a.ldt, 8));
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const int64_t ctas = (a.n * segs + kRowWarps - 1) / kRowWarps;
  auto* k = fp8 ? (vec ? k_embed<true, true> : k_embed<false, true>) : (vec ? k_embed<true, false> : k_embed<false, false>);
  launch_after(k, unsigned(ctas), 32 * kRowWarps, 0, s, a.table, a.tscale, a.rows, a.cols, a.ldt, a.ids, a.id_bits, a.n, a.scale,
                                              static_cast<__nv_bfloat16*>(a.out), a.ldo, segs);
  return check("bq_embed");
}

size_t embed_grad_bytes(int64_t n, int64_t cols) { return embed_grad_plan(n, cols).bytes; }

namespace {

template <bool VEC, typename Out>
int embed_rows(const EmbedRows& a, int pieces, Out* out, cudaStream_t s) {
  const unsigned ctas = unsigned(pieces) * unsigned(a.groups);
  launch_after(k_embed_rows<VEC, Out>, ctas, 32 * kRowWarps, 0, s, a, out);
  if (int rc = check("bq_embed_grad (rows)")) return rc;
  if (pieces < 2) return BQ_OK;  // no run crosses a piece's end
  launch_after(k_embed_join<VEC, Out>, ctas, 32 * kRowWarps, 0, s, a, out);
  return check("bq_embed_grad (join)");
}

}  // namespace

int launch_embed_grad(const EmbedGradArgs& g, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const EmbedGradPlan p = embed_grad_plan(g.n, g.cols);
  auto* w = static_cast<unsigned char*>(ws);
  auto* b0 = reinterpret_cast<uint2*>(w + p.off_b0);
  auto* b1 = reinterpret_cast<uint2*>(w + p.off_b1);
  const bool f32 = g.out_kind == BQ_ROWS_FP32;
  const int size = f32 ? 4 : 2;
  const bool vec = g.cols % 8 == 0 && vec_ok(g.dy, g.ld_dy, 8) && vec_ok(g.out, g.ldo, 16 / size);
  const int passes = (bits_of(g.rows) + kDigit - 1) / kDigit;
  const int n = int(g.n);
  EmbedRows a;
  a.sorted = n <= kChunkTokens || !(passes & 1) ? b0 : b1;
  a.dy = static_cast<const __nv_bfloat16*>(g.dy);
  a.sums = reinterpret_cast<float*>(w + p.off_sums);
  a.ld = g.ld_dy, a.rows = g.rows, a.ldo = g.ldo, a.n = n, a.cols = g.cols, a.ldp = p.ldp;
  a.accumulate = g.accumulate, a.scale = g.scale, a.piece = piece_of(g.n);
  a.groups = (g.cols + kRowWarps * kSpan - 1) / (kRowWarps * kSpan);
  if (int64_t(p.pieces) * a.groups > 0x3FFFFFFF) return set_error(BQ_EINVAL, "bq_embed_grad: batch too large");
  ZeroRows z;
  z.out = static_cast<unsigned char*>(g.out);
  z.rows = g.rows, z.pitch = g.ldo * size, z.row_bytes = g.cols * size;
  const int64_t share = n <= kChunkTokens ? 0 : g.rows * z.row_bytes / (int64_t(sm_count()) * 8);
  z.each = int(std::min<int64_t>(kZeroRows, std::max<int64_t>(1, std::max<int64_t>(kZeroMin, share) / z.row_bytes)));
  z.word = vec_ok(g.out, g.ldo, 16 / size) && z.row_bytes % 16 == 0 ? 16 : size;
  const unsigned zeros = g.accumulate ? 0u : unsigned((g.rows + z.each - 1) / z.each);
  if (n <= kFewTokens) {
    const unsigned ctas = unsigned(n * a.groups) + zeros;
    if (f32)
      launch_after(vec ? k_embed_few<true, float> : k_embed_few<false, float>, ctas, 32 * kRowWarps, 0, s, a, g.ids,
                   g.id_bits, z, static_cast<float*>(g.out));
    else
      launch_after(vec ? k_embed_few<true, __nv_bfloat16> : k_embed_few<false, __nv_bfloat16>, ctas, 32 * kRowWarps, 0, s,
                   a, g.ids, g.id_bits, z, static_cast<__nv_bfloat16*>(g.out));
    return check("bq_embed_grad");
  }
  if (n <= kChunkTokens) {
    // (chunks of ids and positions: n rounded up to whole chunks, in the second buffer)
    const int chunks = (n + kChunk - 1) / kChunk;
    auto* key = reinterpret_cast<uint32_t*>(b1);
    auto* pos = key + chunks * kChunk;
    launch_after(k_embed_chunks, unsigned(chunks) + zeros, kChunk, 0, s, g.ids, g.id_bits, n, int(g.rows), key, pos, z);
    if (int rc = check("bq_embed_grad (chunks)")) return rc;
    launch_after(k_embed_place, unsigned((chunks * kChunk + kPlaceEach - 1) / kPlaceEach), 4 * kPlaceEach, 0, s,
                 static_cast<const uint32_t*>(key), static_cast<const uint32_t*>(pos), n, b0);
  } else {
    launch_after(k_embed_sort, (kSortCtas + zeros + kSortCtas - 1) / kSortCtas * kSortCtas, kSortThreads, 0, s, g.ids,
                 g.id_bits, n, int(g.rows), passes, b0, b1, z);
  }
  if (int rc = check("bq_embed_grad (sort)")) return rc;
  if (f32) {
    auto* out = static_cast<float*>(g.out);
    return vec ? embed_rows<true>(a, p.pieces, out, s) : embed_rows<false>(a, p.pieces, out, s);
  }
  auto* out = static_cast<__nv_bfloat16*>(g.out);
  return vec ? embed_rows<true>(a, p.pieces, out, s) : embed_rows<false>(a, p.pieces, out, s);
}

namespace {

// the ring kernels' shared-memory attribute, set once per device
int ring_attrs() {
  static OncePerDevice once;
  return once.run(current_device(), [] {
    const void* kernels[] = {reinterpret_cast<const void*>(k_norm_many<1>), reinterpret_cast<const void*>(k_norm_many<2>),
                             reinterpret_cast<const void*>(k_norm_many<4>),
                             reinterpret_cast<const void*>(k_norm_grad_many<1>),
                             reinterpret_cast<const void*>(k_norm_grad_many<2>)};
    for (const void* k : kernels)
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
        return check("bq_rmsnorm (shared memory attribute)");
    return int(BQ_OK);
  });
}

}  // namespace

int launch_rmsnorm(const RmsnormArgs& r, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a;
  a.x = static_cast<const __nv_bfloat16*>(r.x);
  a.res = static_cast<const __nv_bfloat16*>(r.residual);
  a.w = static_cast<const __nv_bfloat16*>(r.weight);
  a.h = static_cast<__nv_bfloat16*>(r.h);
  a.y = static_cast<__nv_bfloat16*>(r.y);
  a.codes = r.codes, a.scale = r.code_scale, a.rstd = r.rstd;
  a.ldx = r.ld_x, a.ldr = r.ld_r, a.ldh = r.ld_h, a.ldy = r.ld_y, a.ldc = r.ld_codes, a.lds = r.ld_scale;
  a.eps = r.eps, a.cols = r.cols;
  const bool vec = r.cols % 8 == 0 && vec_ok(r.x, r.ld_x, 8) && (!r.residual || vec_ok(r.residual, r.ld_r, 8)) &&
                   aligned16(r.weight) && (!r.h || vec_ok(r.h, r.ld_h, 8)) && (!r.y || vec_ok(r.y, r.ld_y, 8)) &&
                   (!r.codes || ((reinterpret_cast<uintptr_t>(r.codes) & 7) == 0 && r.ld_codes % 8 == 0));
  int warps, vpt;
  norm_shape(r.cols, vec, &warps, &vpt);
  if (vec && vpt <= 4) {
    const int row = (r.residual ? 2 : 1) * vpt * warps * 512;
    const Ring ring = ring_of(warps, row, r.n, vpt <= 2 ? 1024 : 512, 32);
    if (ring.depth) {
      auto* many = vpt == 1 ? k_norm_many<1> : vpt == 2 ? k_norm_many<2> : k_norm_many<4>;
      if (int rc = ring_attrs()) return rc;
      const int64_t most = int64_t(sm_count()) * ring.per_sm, each = (r.n + most - 1) / most;
      launch_after(many, unsigned((r.n + each - 1) / each), 32 * warps, size_t(ring.depth * row), s, a, r.n, ring.depth);
      return check("bq_rmsnorm");
    }
  }
  auto* k = vec ? (vpt == 1 ? k_norm<true, 1> : vpt == 2 ? k_norm<true, 2> : vpt == 4 ? k_norm<true, 4> : k_norm<true, 8>)
                : (vpt == 1   ? k_norm<false, 1>
                   : vpt == 2 ? k_norm<false, 2>
                   : vpt == 4 ? k_norm<false, 4>
                              : k_norm<false, 8>);
  launch_after(k, unsigned(r.n), 32 * warps, 0, s, a);
  return check("bq_rmsnorm");
}

// pad: the codes' rows may be written up to the next multiple of 8
int launch_quant_rows(const void* x, int64_t ldx, int64_t n, int cols, uint8_t* codes, int64_t ldc, float* scale,
                      int64_t lds, bool pad, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool in = cols % 8 == 0 && vec_ok(x, ldx, 8);
  const bool out = (pad || cols % 8 == 0) && (reinterpret_cast<uintptr_t>(codes) & 7) == 0 && ldc % 8 == 0;
  // four spans a warp share one division pass (8192 x 14336: 57 us, 75 with one); one
  // where that would not give every scheduler a warp
  const int spans = (cols + kSpan - 1) / kSpan;
  const int each = n * ((spans + 3) / 4) >= int64_t(sm_count()) * 4 ? 4 : 1;
  const int segs = (spans + each - 1) / each;
  const int64_t ctas = (n * segs + kRowWarps - 1) / kRowWarps;
  auto* k = each == 4 ? (!out ? k_quant_rows<false, false, 4> : in ? k_quant_rows<true, true, 4> : k_quant_rows<false, true, 4>)
                      : (!out ? k_quant_rows<false, false, 1> : in ? k_quant_rows<true, true, 1> : k_quant_rows<false, true, 1>);
  launch_after(k, unsigned(ctas), 32 * kRowWarps, 0, s, static_cast<const __nv_bfloat16*>(x), ldx, n, cols, codes, ldc,
               scale, lds, segs);
  return check("bq_quant_rows_fp8");
}

int launch_dw_inputs(const uint8_t* codes, int64_t ldc, const float* scale, int64_t lds, int64_t n, int cols, void* x_out,
                     int64_t ldo, const void* dy, int64_t ldy, int rows, void* dy_out, int64_t ldyo, void* stream) {
  DwInputs a;
  a.codes = codes, a.scale = scale, a.dy = static_cast<const __nv_bfloat16*>(dy);
  a.x_out = static_cast<__nv_bfloat16*>(x_out), a.dy_out = static_cast<__nv_bfloat16*>(dy_out);
  a.ldc = ldc, a.lds = lds, a.ldo = ldo, a.ldy = ldy, a.ldyo = ldyo;
  a.cols = cols, a.rows = rows;
  a.x_spans = (cols + kSpan - 1) / kSpan, a.y_spans = (rows + kSpan - 1) / kSpan;
  a.x_items = n * a.x_spans, a.items = a.x_items + (dy ? n * a.y_spans : 0);
  launch_after(k_dw_inputs, unsigned((a.items + kRowWarps - 1) / kRowWarps), 32 * kRowWarps, 0,
               static_cast<cudaStream_t>(stream), a);
  return check("bq_linear_fp8_dw (inputs)");
}

// By the times of 1 to 128 tokens and 512 x 512 to 14336 x 4096.  512 x 512, 16 tokens: 4.4 us
// here, 6.5 on the tensor cores; 32: 7.2 and 6.8.  2880 x 4096, 1 token: 6.6 and 9.6; 16: 13.6
// and 10.2.  14336 x 4096, 1 token: 26.5 and 23.3.
bool dw_few(int64_t n, int64_t rows, int64_t cols) {
  const int64_t tiles = ((rows + kFewRows - 1) / kFewRows) * ((cols + kFewCols - 1) / kFewCols), sms = sm_count();
  const int64_t pairs = ((rows + 255) / 256) * ((cols + 255) / 256), waves = (pairs + sms / 2 - 1) / (sms / 2);
  return 2.0 + double(rows) * double(cols) / 3e6 + 0.12 * double(n) * double((tiles + sms - 1) / sms) <
         5.0 + 1.6 * double(waves) + 0.3 * double(n / 64);
}

int launch_dw_few(const void* dy, int64_t ld_dy, const uint8_t* codes, int64_t ldc, const float* scale, int64_t lds,
                  int n, int rows, int cols, void* dw, int64_t ld_dw, int accumulate, void* stream) {
  const int64_t tiles = int64_t((rows + kFewRows - 1) / kFewRows) * ((cols + kFewCols - 1) / kFewCols);
  launch_after(k_dw_few, unsigned(tiles), 256, 0, static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(dy),
               ld_dy, codes, ldc, scale, lds, n, rows, cols, static_cast<__nv_bfloat16*>(dw), ld_dw, accumulate);
  return check("bq_linear_fp8_dw");
}

size_t rmsnorm_grad_bytes(int64_t n, int64_t cols) {
  const size_t ldp = size_t((cols + kSpan - 1) / kSpan * kSpan);
  const int ctas = norm_grad_plan(n, int(cols), 2, false).ctas;  // (whatever the operands)
  return std::max<size_t>(256, size_t(ctas) * ldp * 4);
}

int launch_rmsnorm_grad(const RmsnormGradArgs& r, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormGradArgs a;
  a.dy = static_cast<const __nv_bfloat16*>(r.dy);
  a.h = static_cast<const __nv_bfloat16*>(r.h);
  a.w = static_cast<const __nv_bfloat16*>(r.weight);
  a.dh = static_cast<const __nv_bfloat16*>(r.dh);
  a.rstd = r.rstd;
  a.dx = static_cast<__nv_bfloat16*>(r.dx);
  a.part = static_cast<float*>(ws);
  a.ld_dy = r.ld_dy, a.ld_h = r.ld_h, a.ld_dh = r.ld_dh, a.ld_dx = r.ld_dx, a.n = r.n;
  a.cols = r.cols, a.ldp = (r.cols + kSpan - 1) / kSpan * kSpan;
  const bool vec = r.cols % 8 == 0 && vec_ok(r.dy, r.ld_dy, 8) && vec_ok(r.h, r.ld_h, 8) && aligned16(r.weight) &&
                   (!r.dh || vec_ok(r.dh, r.ld_dh, 8)) && vec_ok(r.dx, r.ld_dx, 8);
  const NormGradPlan p = norm_grad_plan(r.n, r.cols, r.dh ? 3 : 2, vec);
  if (p.depth) {
    if (int rc = ring_attrs()) return rc;
    auto* k = p.vpt == 1 ? k_norm_grad_many<1> : k_norm_grad_many<2>;
    launch_after(k, unsigned(p.ctas), 32 * p.warps, size_t(p.smem), s, a, p.depth);
  } else if (p.ctas > 0) {
    auto* k = vec ? (p.vpt == 1 ? k_norm_grad<true, 1> : p.vpt == 2 ? k_norm_grad<true, 2> : k_norm_grad<true, 8>)
                  : (p.vpt == 1 ? k_norm_grad<false, 1> : p.vpt == 2 ? k_norm_grad<false, 2> : k_norm_grad<false, 8>);
    launch_after(k, unsigned(p.ctas), 32 * p.warps, 0, s, a);
  }
  if (int rc = check("bq_rmsnorm_grad")) return rc;
  const unsigned g = unsigned((r.cols + 31) / 32);
  const float* part = a.part;
  if (r.dw_kind == BQ_ROWS_FP32)
    launch_after(k_norm_dw<float>, g, 1024, 0, s, part, p.ctas, a.ldp, r.cols, r.accumulate, static_cast<float*>(r.dw));
  else
    launch_after(k_norm_dw<__nv_bfloat16>, g, 1024, 0, s, part, p.ctas, a.ldp, r.cols, r.accumulate,
                 static_cast<__nv_bfloat16*>(r.dw));
  return check("bq_rmsnorm_grad (dw)");
}

}  // namespace bq
