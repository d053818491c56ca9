// The tiles of products on CTA pairs: their shape, their epilogue warps' staging of 16-bit
// outputs and the launch of clusters, shared by the FP8 projections (linear_fp8.cu) and
// the losses over an FP8 head (loss_fp8.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "umma_ptx.h"

namespace bq {

constexpr int BK = 128;  // a k-block: one scale group, 128 bytes of codes
constexpr int PM = 256, PN = 256, kBand = 8;    // a pair's tile of out, row blocks of a band
constexpr int HALF_STAGE = 128 * BK;            // 16 KB
constexpr int PSTAGE_BYTES = 2 * HALF_STAGE;
// Sixteen epilogue warps, four per tensor-memory lane quarter: part p of a quarter
// reads columns 64p .. 64p + 63 of every accumulator.  Five warpgroups with TMA (warp
// 0) and MMA (warp 1); of the launch's 640 x 96 registers the first group keeps 32 a
// thread and the epilogue takes 112.
constexpr int PEPI = 16, PCOLS = PN / 4;
constexpr int PAIR_THREADS = 128 + 32 * PEPI;
constexpr int kRegsLaunch = 96, kRegsIssue = 32, kRegsEpilogue = 112;
static_assert(128 * kRegsIssue + 32 * PEPI * kRegsEpilogue <= PAIR_THREADS * kRegsLaunch, "register split");
constexpr int OUT_BOX = 32 * 64;                // 32 rows x 32 bf16 of out, one a warp
constexpr int kPairTmem = 2 * PN;
constexpr int DK = 64;                          // summed rows of a k-block of 16-bit operands
constexpr int CHUNK = DK * 128;                 // 64 of them x 64 columns: 8 KB, two an operand
constexpr int DW_STAGES = 5, DW_BOX = 32 * 128;  // (a warp's staging of out: 32 rows x 64 values)
constexpr int DW_SMEM = 1024 + DW_STAGES * PSTAGE_BYTES + PEPI * DW_BOX;

// acc += f * r
template <int N>
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t* r, float f) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 o = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), make_float2(f, f),
                                make_float2(acc[j], acc[j + 1]));
    acc[j] = o.x;
    acc[j + 1] = o.y;
  }
}

// `bytes` (0 to 16, the rest zeros) to 16-byte aligned shared memory
__device__ __forceinline__ void copy16_clipped(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// arrives on the barrier (whose count includes it) when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A warp's box of out, 32 rows x COLS 16-bit values (32 or 64) in shared memory, swizzled as its store
// reads it: 16-byte word c of row r at word c ^ ((r >> 1) & 3), or c ^ (r & 7)
template <int COLS>
__device__ __forceinline__ uint32_t box_word(uint32_t box, int r, int c) {
  return box + 2u * COLS * uint32_t(r) + 16u * uint32_t(COLS == 32 ? c ^ ((r >> 1) & 3) : c ^ (r & 7));
}

__device__ __forceinline__ uint32_t two16(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t two16(float a, float b, __half) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// v: the lane's row, as T
template <int COLS, typename T = __nv_bfloat16>
__device__ __forceinline__ void put_box(const float* v, uint32_t box, int lane) {
#pragma unroll
  for (int c = 0; c < COLS / 8; ++c) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = two16(v[8 * c + 2 * e], v[8 * c + 2 * e + 1], T());
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box_word<COLS>(box, lane, c)), "r"(o[0]), "r"(o[1]),
                 "r"(o[2]), "r"(o[3])
                 : "memory");
  }
}

// the box by plain stores of `bytes` (8, 4 or 2, as out's rows are aligned), a row's pieces
// beside one another in the warp, eight loads before their stores
template <int COLS, int BYTES>
__device__ __forceinline__ void store_pieces(__nv_bfloat16* out, int64_t ldo, int rows, int cols, int row0, int c0,
                                             uint32_t box, int lane) {
  constexpr int N = BYTES / 2, LANES = COLS / N < 32 ? COLS / N : 32, EACH = 32 / LANES;  // lanes a row, rows at once
#pragma unroll
  for (int k = 0; k < COLS; k += LANES * N) {
    const int c = k + lane % LANES * N, left = cols - c0 - c;
#pragma unroll 1
    for (int r0 = lane / LANES; r0 < 32; r0 += 8 * EACH) {
      uint32_t v[8][BYTES == 8 ? 2 : 1];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (r0 + e * EACH >= 32) continue;
        const uint32_t at = box_word<COLS>(box, r0 + e * EACH, c >> 3) + 2u * uint32_t(c & 7);
        if constexpr (BYTES == 8)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[e][0]), "=r"(v[e][1]) : "r"(at) : "memory");
        else if constexpr (BYTES == 4)
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[e][0]) : "r"(at) : "memory");
        else
          asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v[e][0]) : "r"(at) : "memory");
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = r0 + e * EACH;
        if (r >= 32 || row0 + r >= rows || left <= 0) continue;
        __nv_bfloat16* o = out + int64_t(row0 + r) * ldo + c0 + c;
        if (left >= N) {
          if constexpr (BYTES == 8)
            *reinterpret_cast<uint2*>(o) = make_uint2(v[e][0], v[e][1]);
          else if constexpr (BYTES == 4)
            *reinterpret_cast<uint32_t*>(o) = v[e][0];
          else
            *reinterpret_cast<uint16_t*>(o) = uint16_t(v[e][0]);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j < left) reinterpret_cast<uint16_t*>(o)[j] = uint16_t(v[e][j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  }
}

// the box to out's row0.., c0.., clipped to rows x cols: by TMA where out's rows are 16-byte
// aligned (`bytes`, as store_bytes has it)
template <int COLS>
__device__ __forceinline__ void store_box(__nv_bfloat16* out, int64_t ldo, int rows, int cols, int bytes,
                                          const CUtensorMap* map, int row0, int c0, uint32_t box, int lane) {
  if (bytes == 16) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0 && row0 < rows && c0 < cols) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(c0), "r"(row0), "r"(box)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  } else {
    __syncwarp();
    if (bytes == 8)
      store_pieces<COLS, 8>(out, ldo, rows, cols, row0, c0, box, lane);
    else if (bytes == 4)
      store_pieces<COLS, 4>(out, ldo, rows, cols, row0, c0, box, lane);
    else
      store_pieces<COLS, 2>(out, ldo, rows, cols, row0, c0, box, lane);
    __syncwarp();
  }
}

// the widest store that out's rows are aligned to.  A copy by TMA clips rows at whole 16-byte
// words only: where they end inside one it would write zeros past their end
inline int store_bytes(const void* out, int64_t ldo, int cols) {
  int bytes = cols % 8 ? 8 : 16;
  while (bytes > 2 && (ldo * 2 % bytes || reinterpret_cast<uintptr_t>(out) % bytes)) bytes /= 2;
  return bytes;
}

// A share's values as the epilogue warps hold them: float4 j of lane l (columns 4j .. of its
// row) at 32 j + l of warp w's 512, so that every store is whole lines (by rows, 16 bytes a
// lane, the same stores took 4 us longer).
__device__ __forceinline__ int64_t share_at(int t, int rank, int w) {
  return ((int64_t(t) * 2 + rank) * PEPI + w) * 512;
}

// linear_fp8.cu: clusters of k = 1 .. 8 CTAs that fit the device at once; a launch of clusters
// with dependent launch, its failure recorded for `what`
const int* cluster_slots();
int launch_clusters(const char* what, const void* kernel, int clusters, int size, int threads, int smem, void** args,
                    cudaStream_t s);

}  // namespace bq
