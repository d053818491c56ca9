// FP8 projections on GB300 tensor cores (sm_103a): out = X W^T and out = X W, X
// FP8 rows with one scale per 128 summed values, W the E4M3 codes of a gathered
// parameter with one scale per 128 x 128 tile.
//
// Per 128 of the summed index (a k-block) the code products are one tensor-core
// sum in fp32, which starts at zero; the epilogue warps read it from tensor memory
// and add it to fp32 registers times the block's two scales.  Two tensor-memory
// accumulators alternate, so that reading one overlaps the products of the next.
// (Scaling per k-block is what the format asks for: the scales are arbitrary fp32
// values, so they cannot be handed to the tensor core, whose own block scales are
// powers of two per 32 values.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "bq_internal.h"
#include "row_ops.h"
#include "tmem_ptx.h"
#include "umma_ptx.h"

namespace bq {
namespace {

int check(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BQ_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return BQ_OK;
}

constexpr int BK = 128;  // a k-block: one scale group, 128 bytes of codes
constexpr int BM = 128, BN = 128;
constexpr int EPI_WARPS = 8;                   // two per tensor-memory lane quarter, each half of a tile's columns
constexpr int THREADS = 64 + 32 * EPI_WARPS;   // warp 0 TMA, warp 1 MMA + TMEM, then the epilogue
constexpr int B_STAGE = BN * BK;
constexpr int kMaxStages = 8;
constexpr int kPartPitch = BN + 1;             // floats of a row of a split's partial tile in shared memory
constexpr int kTmemCols = 2 * BN;
constexpr int kSmem = 112 * 1024;               // dynamic shared memory at most: two CTAs per SM

// Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B E4M3 (bits
// 7-9 and 10-12 = 0), A K-major, B major in bit 16, N >> 3 in bits 17-22, M >> 4 in
// bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n, int b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct LinArgs {
  const float *xs, *ws;  // scales of X [groups][ld_xs] and of W's tiles
  __nv_bfloat16* out;
  int64_t ld_xs, ldo;
  int n, width;          // rows and columns of out
  int red;               // summed index
  int tile_cols;         // W's tiles in a row of tiles
  int transposed;        // 0: out = X W^T, 1: out = X W
  int split, stages;     // CTAs of a cluster that share a tile's k-blocks; pipeline stages
  int a_rows;            // rows of X that a stage holds (a multiple of 8, <= 128)
  int* status;
};

// One 128 x 128 tile of out per cluster; CTA r of the cluster's `split` sums its
// share of the k-blocks, and the shares are added in order through distributed
// shared memory.
__global__ void __launch_bounds__(THREADS, 2)
    k_linear(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const LinArgs g) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * kMaxStages + 2 + b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank());
  const int tile = int(blockIdx.x) / g.split;
  const int nt = (g.width + BN - 1) / BN;
  const int m0 = (tile / nt) * BM, n0 = (tile % nt) * BN;
  const int nk = (g.red + BK - 1) / BK;
  const int k0 = int(int64_t(nk) * rank / g.split), k1 = int(int64_t(nk) * (rank + 1) / g.split);
  const uint32_t b_base = base, a_base = base + uint32_t(g.stages) * B_STAGE;
  const uint32_t a_stage = uint32_t(g.a_rows) * BK;
  // lane quarters with rows of out: only their warps read the accumulators
  const int quarters = min(4, (g.n - m0 + 31) / 32);

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), uint32_t(2 * quarters));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  float acc[BN / 2];
#pragma unroll
  for (int j = 0; j < BN / 2; ++j) acc[j] = 0.f;
  const int q = warp & 3, half = (warp - 2) >> 2;  // epilogue warps

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer
    int it = 0;
    for (int kb = k0; kb < k1; ++kb, ++it) {
      const int s = it % g.stages;
      if (!mbar_wait(empty_bar(s), uint32_t((it / g.stages) & 1) ^ 1u, g.status, 21)) break;
      mbar_expect_tx(full_bar(s), a_stage + B_STAGE);
      tma_load_2d(a_base + uint32_t(s) * a_stage, &tmX, kb * BK, m0, full_bar(s));
      if (g.transposed)
        tma_load_2d(b_base + uint32_t(s) * B_STAGE, &tmW, n0, kb * BK, full_bar(s));
      else
        tma_load_2d(b_base + uint32_t(s) * B_STAGE, &tmW, kb * BK, n0, full_bar(s));
    }
    // drain: the last load issued to each stage has landed before this CTA can exit
    for (int d = max(0, it - g.stages); d < it; ++d)
      mbar_wait(full_bar(d % g.stages), uint32_t((d / g.stages) & 1), g.status, 22);
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer
    const uint32_t id = idesc_e4m3(BM, BN, g.transposed);
    int it = 0;
    for (int kb = k0; kb < k1; ++kb, ++it) {
      const int s = it % g.stages, buf = it & 1;
      if (it >= 2 && !mbar_wait(tempty_bar(buf), uint32_t((it >> 1) & 1) ^ 1u, g.status, 23)) break;
      if (!mbar_wait(full_bar(s), uint32_t((it / g.stages) & 1), g.status, 24)) break;
      tc_fence_after();
      const uint32_t a_addr = a_base + uint32_t(s) * a_stage, b_addr = b_base + uint32_t(s) * B_STAGE;
#pragma unroll
      for (int kk = 0; kk < BK / 32; ++kk) {
        // K-major: 32-code k slices 32 bytes apart; MN-major: 32 k rows of 128 bytes apart
        const uint64_t ad = sdesc(a_addr + 32u * kk, 16, 1024);
        const uint64_t bd = g.transposed ? sdesc(b_addr + 32u * 128u * kk, BK * 128, 1024)
                                         : sdesc(b_addr + 32u * kk, 16, 1024);
        mma_e4m3(tmem + uint32_t(buf) * BN, ad, bd, id, kk != 0 ? 1u : 0u);
      }
      mma_commit(empty_bar(s));
      mma_commit(tfull_bar(buf));
    }
    // every product issued here has finished before the accumulators are freed
    if (it > 0) mbar_wait(tfull_bar((it - 1) & 1), uint32_t(((it - 1) >> 1) & 1), g.status, 26);
  } else if (warp >= 2 && q < quarters) {
    // ---------------- scaled accumulation
    const int row = m0 + 32 * q + lane;
    const float* xs = g.xs + row;
    // the tile's 128 columns of out lie in one row (transposed: column) of W's tiles
    const float* ws = g.transposed ? g.ws + (n0 >> 7) : g.ws + int64_t(n0 >> 7) * g.tile_cols;
    const int64_t ws_step = g.transposed ? g.tile_cols : 1;
    const bool on = row < g.n;
    float f = 0.f;
    if (k0 < k1 && on) f = __ldg(xs + int64_t(k0) * g.ld_xs) * __ldg(ws + k0 * ws_step);
    int it = 0;
    for (int kb = k0; kb < k1; ++kb, ++it) {
      const int buf = it & 1;
      const float fk = f;
      if (kb + 1 < k1 && on) f = __ldg(xs + int64_t(kb + 1) * g.ld_xs) * __ldg(ws + (kb + 1) * ws_step);
      if (!mbar_wait(tfull_bar(buf), uint32_t((it >> 1) & 1), g.status, 25)) break;
      tc_fence_after();
      const uint32_t at = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf) * BN + uint32_t(half) * (BN / 2);
#pragma unroll
      for (int j0 = 0; j0 < BN / 2; j0 += 32) {
        uint32_t r[32];
        tmem_ld32(at + uint32_t(j0), r);
        if (j0 + 32 == BN / 2) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(tempty_bar(buf));
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 o = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                      make_float2(fk, fk), make_float2(acc[j0 + j], acc[j0 + j + 1]));
          acc[j0 + j] = o.x;
          acc[j0 + j + 1] = o.y;
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();  // the stages are free: every copy has landed and every product is done
  float* part = reinterpret_cast<float*>(gbase);
  if (warp >= 2 && q < quarters) {
    float* prow = part + (32 * q + lane) * kPartPitch + half * (BN / 2);
#pragma unroll
    for (int j = 0; j < BN / 2; ++j) prow[j] = acc[j];
  }
  cluster_sync();  // (every thread) the cluster's partial tiles are written
  const int rows = min(BM, g.n - m0), cols = min(BN, g.width - n0);
  // each CTA finishes its share of the tile's rows: lane l columns l, l + 32, ...
  const uint32_t part0 = smem_addr(part);
  for (int r = rank * (THREADS / 32) + warp; r < rows; r += g.split * (THREADS / 32)) {
    float v[BN / 32];
#pragma unroll
    for (int j = 0; j < BN / 32; ++j) v[j] = 0.f;
    for (int c = 0; c < g.split; ++c) {
      const uint32_t at = map_rank(part0, uint32_t(c)) + 4u * uint32_t(r * kPartPitch + lane);
#pragma unroll
      for (int j = 0; j < BN / 32; ++j) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at + 128u * j) : "memory");
        v[j] += x;
      }
    }
    __nv_bfloat16* o = g.out + int64_t(m0 + r) * g.ldo + n0;
#pragma unroll
    for (int j = 0; j < BN / 32; ++j)
      if (lane + 32 * j < cols) o[lane + 32 * j] = __float2bfloat16_rn(v[j]);
  }
  tc_fence_before();
  cluster_sync();  // a partial tile outlives its readers; tensor memory its users
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int launch_linear_fp8(const LinearArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int width = a.transposed ? a.cols : a.rows, red = a.transposed ? a.rows : a.cols;
  LinArgs g;
  g.xs = a.x_scale, g.ws = a.w_scale, g.out = static_cast<__nv_bfloat16*>(a.out);
  g.ld_xs = a.ld_xs, g.ldo = a.ldo, g.n = int(a.n), g.width = width, g.red = red;
  g.tile_cols = (a.cols + 127) / 128, g.transposed = a.transposed, g.status = a.status;
  g.a_rows = int(std::min<int64_t>(BM, (a.n + 7) / 8 * 8));
  const int64_t tiles = ((a.n + BM - 1) / BM) * ((width + BN - 1) / BN);
  const int nk = (red + BK - 1) / BK;
  // two CTAs share an SM.  The X stages come last, and a product reads 128 rows of
  // the last one whatever it holds: what follows it is spare shared memory
  const int stage = B_STAGE + g.a_rows * BK, spare = (BM - g.a_rows) * BK;
  const int part = BM * kPartPitch * 4;
  g.stages = std::min(kMaxStages, (kSmem - 1024 - spare) / stage);
  // k-blocks are split while the tiles leave resident CTAs idle and a share keeps
  // at least four
  g.split = 1;
  while (g.split < 8 && tiles * g.split * 2 <= int64_t(sm_count()) * 2 && nk / (g.split * 2) >= 4) g.split *= 2;
  CUtensorMap tx, tw;
  if (int rc = encode_map_codes(&tx, a.x, red, a.n, a.ldx, g.a_rows)) return rc;
  if (int rc = encode_map_codes(&tw, a.w, a.cols, a.rows, a.ldw, 128)) return rc;
  const int smem = 1024 + std::max(part, g.stages * stage + spare);
  if (once_per_device(kOnceLinearAttr) &&
      cudaFuncSetAttribute(k_linear, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return check("bq_linear_fp8 (shared memory attribute)");
  if (tiles * g.split > 0x7FFFFFFF) return set_error(BQ_EINVAL, "bq_linear_fp8: too many tiles");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(g.split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(tiles * g.split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_linear, tx, tw, g) != cudaSuccess) return check("bq_linear_fp8");
  return check("bq_linear_fp8");
}

}  // namespace bq
