// bf16 and E4M3 conversions, packed fp32 pairs and block scales, shared by the
// DBuffer step and the layer operators.  Every fp32 operation is an explicit
// round-to-nearest intrinsic, so the results do not depend on the flags of the
// file that includes this.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bq {

__device__ __forceinline__ float bf16f(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

__device__ __forceinline__ uint32_t f2bf(float x) {
  return uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(x)));
}

// Blackwell's packed fp32 pair arithmetic: each component is rounded exactly
// like the scalar round-to-nearest operation.  A packed add takes no product as
// an operand anywhere below: ptxas contracts a packed multiply feeding a packed
// add into a fused multiply-add even when both carry an explicit .rn, so every
// multiply-then-add is written as the explicit fused operation the contract
// specifies.
__device__ __forceinline__ float2 dup(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }  // operands never products
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// max of three floats; a NaN operand gives NaN (so a NaN in a block reaches its
// scale, as a maximum over the raw bit patterns would)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Block scale from an absmax (fp32 bits; all values >= 0 so bit order == value
// order): stored scale s = amax/qmax, reciprocal r = qmax/amax (one division each
// per block).  mode 0: s == 0 -> zero codes; 1: codes from x*r; 2: r overflowed
// (tiny amax) -> codes from x/s.
struct QScale {
  float s, r;
  int mode;
};

__device__ __forceinline__ QScale qscale(uint32_t amax_bits, float qmax) {
  const float a = __uint_as_float(amax_bits);
  QScale q;
  q.s = __fdiv_rn(a, qmax);
  q.r = __fdiv_rn(qmax, a);
  q.mode = q.s == 0.f ? 0 : (isinf(q.r) ? 2 : 1);
  return q;
}

// 8 E4M3 codes (round to nearest even, saturating); scale 0 keeps each sign
__device__ __forceinline__ uint2 codes_e4m3(const float* x, const QScale& q) {
  uint32_t w[4];
  if (q.mode == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = ((__float_as_uint(x[2 * i]) >> 24) & 0x80u) | ((__float_as_uint(x[2 * i + 1]) >> 16) & 0x8000u);
  } else if (q.mode == 1) {
    const float2 r = dup(q.r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = uint32_t(__nv_cvt_float2_to_fp8x2(mul2(make_float2(x[2 * i], x[2 * i + 1]), r), __NV_SATFINITE, __NV_E4M3));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], q.s), __fdiv_rn(x[2 * i + 1], q.s)),
                                               __NV_SATFINITE, __NV_E4M3));
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace bq
