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
#include <mutex>
#include <string>

#include "bq_internal.h"
#include "once.h"
#include "pdl.h"
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
constexpr int kAhead = 4;                      // k-blocks from a scale's load to its use
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

struct LinArgs {
  const float *xs, *ws;  // scales of X [groups][ld_xs] and of W's tiles
  __nv_bfloat16* out;
  int64_t ld_xs, ldo;
  int n, width;          // rows and columns of out
  int red;               // summed index
  int tile_cols;         // W's tiles in a row of tiles
  int split, stages;     // CTAs of a cluster that share a tile's k-blocks; pipeline stages
  int a_rows;            // rows of X that a stage holds (a multiple of 8, <= 128)
  int bytes;             // of a store into out (store_bytes)
  int* status;
};

// One 128 x 128 tile of out per cluster; CTA r of the cluster's `split` sums its
// share of the k-blocks, and the shares are added in order through distributed
// shared memory.  For few rows, where the weight's bytes and then the start of a CTA count:
// 1 row of 8192 x 8192 takes 14.2 us (4.7 TB/s; its bytes alone are 9.9), 333 rows of 2880 x
// 4096 take 11.7 (0.6 us of set-up, 0.9 to the first product, 16 k-blocks at 0.35 to 0.44, 3 for
// the join and the stores).
template <bool TRANS>
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
  const int k0 = int(int64_t(nk) * rank / g.split), blocks = int(int64_t(nk) * (rank + 1) / g.split) - k0;
  const uint32_t b_base = base, a_base = base + uint32_t(g.stages) * B_STAGE;
  const uint32_t a_stage = uint32_t(g.a_rows) * BK;
  // lane quarters with rows of out: only their warps read the accumulators
  const int quarters = min(4, (g.n - m0 + 31) / 32);

  auto load = [&](int it, int s) {  // one lane: k-block it of this CTA into stage s
    const int kb = k0 + it;
    mbar_expect_tx(full_bar(s), a_stage + B_STAGE);
    if (TRANS)
      tma_load_2d(b_base + uint32_t(s) * B_STAGE, &tmW, n0, kb * BK, full_bar(s));
    else
      tma_load_2d(b_base + uint32_t(s) * B_STAGE, &tmW, kb * BK, n0, full_bar(s));
    tma_load_2d(a_base + uint32_t(s) * a_stage, &tmX, kb * BK, m0, full_bar(s));
  };
  after_previous();
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
    for (int it = 0; it < min(blocks, g.stages); ++it) load(it, it);  // the first stages, before the set-up below
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  next_may_start();
  const uint32_t tmem = tmem_slot;

  float acc[BN / 2];
#pragma unroll
  for (int j = 0; j < BN / 2; ++j) acc[j] = 0.f;
  const int q = warp & 3, half = (warp - 2) >> 2;  // epilogue warps

  // (the issuing warps run whole, one elected lane issues: see k_linear_pair)
  if (warp == 0) {
    // ---------------- TMA producer
    int it = min(blocks, g.stages);
    for (int s = 0, use = 1; it < blocks; ++it) {
      if (!mbar_wait(empty_bar(s), uint32_t(use & 1) ^ 1u, g.status, 21)) break;
      if (elect_one()) load(it, s);
      __syncwarp();
      if (++s == g.stages) s = 0, ++use;
    }
    // drain: the last load issued to each stage has landed before this CTA can exit
    for (int d = max(0, it - g.stages); d < it; ++d)
      mbar_wait(full_bar(d % g.stages), uint32_t((d / g.stages) & 1), g.status, 22);
  } else if (warp == 1) {
    // ---------------- MMA issuer
    const uint32_t id = idesc_e4m3(BM, BN, TRANS ? 1 : 0);
    int it = 0;
    for (int s = 0, use = 0; it < blocks; ++it) {
      const int buf = it & 1;
      if (it >= 2 && !mbar_wait(tempty_bar(buf), uint32_t((it >> 1) & 1) ^ 1u, g.status, 23)) break;
      if (!mbar_wait(full_bar(s), uint32_t(use & 1), g.status, 24)) break;
      tc_fence_after();
      // K-major: 32-code k slices 32 bytes apart; MN-major: 32 k rows of 128 bytes apart
      const uint64_t ad = sdesc(a_base + uint32_t(s) * a_stage, 16, 1024);
      const uint64_t bd = sdesc(b_base + uint32_t(s) * B_STAGE, TRANS ? BK * 128 : 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma_e4m3(tmem + uint32_t(buf) * BN, ad + uint64_t(2 * kk), bd + uint64_t(TRANS ? 256 * kk : 2 * kk), id,
                   kk != 0 ? 1u : 0u);
        mma_commit(empty_bar(s));
        mma_commit(tfull_bar(buf));
      }
      __syncwarp();
      if (++s == g.stages) s = 0, ++use;
    }
    // every product issued here has finished before the accumulators are freed
    if (it > 0) mbar_wait(tfull_bar((it - 1) & 1), uint32_t(((it - 1) >> 1) & 1), g.status, 26);
  } else if (q < quarters) {
    // ---------------- scaled accumulation
    const int row = m0 + 32 * q + lane;
    const bool on = row < g.n;
    const float* xs = g.xs + row + int64_t(k0) * g.ld_xs;
    // the tile's 128 columns of out lie in one row (transposed: column) of W's tiles
    const int64_t ws_step = TRANS ? g.tile_cols : 1;
    const float* ws = (TRANS ? g.ws + (n0 >> 7) : g.ws + int64_t(n0 >> 7) * g.tile_cols) + k0 * ws_step;
    // scales come kAhead blocks before their use (their loads queue behind the stages'
    // copies); W's for 32 blocks at a time, block b in lane b
    float xn[kAhead], wl = 0.f, wn = lane < blocks ? __ldg(ws + lane * ws_step) : 0.f;
#pragma unroll
    for (int b = 0; b < kAhead; ++b) xn[b] = on && b < blocks ? __ldg(xs + b * g.ld_xs) : 0.f;
    bool ok = true;
    for (int it0 = 0; it0 < blocks; it0 += kAhead) {
      if ((it0 & 31) == 0) {
        wl = wn;
        wn = it0 + 32 + lane < blocks ? __ldg(ws + (it0 + 32 + lane) * ws_step) : 0.f;
      }
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        const int it = it0 + b;
        if (it >= blocks) continue;  // (no early exit: its copies of the sums would spill)
        const float f = xn[b] * __shfl_sync(0xFFFFFFFFu, wl, it & 31);
        if (on && it + kAhead < blocks) xn[b] = __ldg(xs + int64_t(it + kAhead) * g.ld_xs);
        const int buf = it & 1;
        ok = ok && mbar_wait(tfull_bar(buf), uint32_t((it >> 1) & 1), g.status, 25);
        tc_fence_after();
        const uint32_t at = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf) * BN + uint32_t(half) * (BN / 2);
#pragma unroll
        for (int j0 = 0; j0 < BN / 2; j0 += 16) {
          uint32_t r[16];
          tmem_ld16_begin(at + uint32_t(j0), r);
          tmem_wait_ld16(r);
          if (j0 + 16 == BN / 2) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(tempty_bar(buf));
          }
          add_scaled<16>(acc + j0, r, f);
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
    if (g.split == 1) {
#pragma unroll
      for (int j = 0; j < BN / 32; ++j) v[j] = part[r * kPartPitch + lane + 32 * j];
    } else {
      for (int c0 = 0; c0 < g.split; c0 += 4) {  // four shares' loads set out together
        float x[4][BN / 32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c0 + c >= g.split) break;
          const uint32_t at = map_rank(part0, uint32_t(c0 + c)) + 4u * uint32_t(r * kPartPitch + lane);
#pragma unroll
          for (int j = 0; j < BN / 32; ++j)
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[c][j]) : "r"(at + 128u * j) : "memory");
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c0 + c < g.split)
#pragma unroll
            for (int j = 0; j < BN / 32; ++j) v[j] += x[c][j];
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

// ---------------------------------------------------------------- CTA pairs
// Large products: pairs of CTAs (cta_group::2, one pair per two SMs) walk 256 x 256
// tiles of out in bands of kBand row blocks.  Each CTA stages its 128 rows of X and its
// 128 columns (W rows, or W columns when transposed) of a k-block; the leader issues
// M = 256 products that read both CTAs' shared memory.  A tile's fp32 sums stay in the
// epilogue warps' registers (64 a thread); its bf16 rows leave through shared memory
// and TMA stores while the next tile's products run.
//
// Two accumulators of N = 256 fill tensor memory: k-block it sums into accumulator it & 1
// while the epilogue reads the other.  A product takes the tensor cores 512 cycles a
// k-block for N = 128 and 192 as well (X's rows, read from shared memory, set its pace), so
// four accumulators of N = 128 took 391 us and 192-column tiles 387 where these took 340
// (8192 rows, 14336 x 4096; 347 since the scales have a ring of their own).
//
// What bounds it: from one product's start to the next on the same accumulator pass about
// 1400 cycles (512 of products, 370 until the epilogue sees them done, 400 to read them and
// add half, 100 until the last arrival starts the next), so a k-block takes 700; and power,
// which holds the clock near 1.7 GHz.  347 us are 2.77 PFLOP/s, in a run of seconds 390 us.
// Without the epilogue's reading and adding the same products and copies take 258 us, at
// 1.5 GHz (twice the rate of a library's bf16 product: 252).
constexpr int PM = 256, PN = 256, PSTAGES = 5, kBand = 8;
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
// X's scales of a k-block (128 rows of this CTA) come through a ring of their own, up to
// SLOTS k-blocks ahead: loads by the epilogue warps themselves would queue behind the
// stages' copies.  Warp 2 copies them with cp.async, four scales a lane, and each CTA has its
// own two barriers a slot: its 32 lanes' copies complete the one, its epilogue warps, when
// they have read the slot, the other.  Every access is of the generic proxy and every
// hand-over a release and an acquire within the CTA, so nothing else has to order a
// slot's readers and its next copy (a bulk copy into a slot that plain loads read would want a
// proxy fence a warp and k-block).  A warp takes its scale before it waits for the products;
// taken a k-block ahead, between the reading of the accumulator and the additions, it cost
// 367 us in place of 347 (8192 rows, 14336 x 4096; spills).
constexpr int SLOTS = 8, SLOT_BYTES = 128 * 4;
constexpr int OFF_OUT = PSTAGES * PSTAGE_BYTES, OFF_SCALES = OFF_OUT + PEPI * OUT_BOX;
constexpr int PAIR_SMEM = 1024 + OFF_SCALES + SLOTS * SLOT_BYTES;
constexpr int kPairTmem = 2 * PN;

// `bytes` (0 to 16, the rest zeros) to 16-byte aligned shared memory
__device__ __forceinline__ void copy16_clipped(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// arrives on the barrier (whose count includes it) when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A warp's box of out, 32 rows x COLS bf16 (32 or 64) in shared memory, swizzled as its store
// reads it: 16-byte word c of row r at word c ^ ((r >> 1) & 3), or c ^ (r & 7)
template <int COLS>
__device__ __forceinline__ uint32_t box_word(uint32_t box, int r, int c) {
  return box + 2u * COLS * uint32_t(r) + 16u * uint32_t(COLS == 32 ? c ^ ((r >> 1) & 3) : c ^ (r & 7));
}

// v: the lane's row
template <int COLS>
__device__ __forceinline__ void put_box(const float* v, uint32_t box, int lane) {
#pragma unroll
  for (int c = 0; c < COLS / 8; ++c) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[8 * c + 2 * e], v[8 * c + 2 * e + 1]);
      o[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
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
int store_bytes(const void* out, int64_t ldo, int cols) {
  int bytes = cols % 8 ? 8 : 16;
  while (bytes > 2 && (ldo * 2 % bytes || reinterpret_cast<uintptr_t>(out) % bytes)) bytes /= 2;
  return bytes;
}

template <bool TRANS>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmO, const LinArgs g) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  __shared__ __align__(8) uint64_t bars[2 * PSTAGES + 4 + 2 * SLOTS];
  __shared__ uint32_t tmem_slot;
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(PSTAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * PSTAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * PSTAGES + 2 + b); };
  auto sfull_bar = [&](int l) { return bar0 + 8u * uint32_t(2 * PSTAGES + 4 + l); };
  auto sempty_bar = [&](int l) { return bar0 + 8u * uint32_t(2 * PSTAGES + 4 + SLOTS + l); };

  const int rank = int(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = (g.n + PM - 1) / PM, nt = (g.width + PN - 1) / PN, ntiles = mt * nt;
  const int nk = (g.red + BK - 1) / BK;
  const int pair = int(blockIdx.x >> 1), npairs = int(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < PSTAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the leader's expect_tx
      mbar_init(empty_bar(s), 1);  // the leader's commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * PEPI);  // the epilogue warps of both CTAs
    }
    for (int l = 0; l < SLOTS; ++l) {
      mbar_init(sfull_bar(l), 32);     // warp 2's lanes
      mbar_init(sempty_bar(l), PEPI);  // this CTA's epilogue warps
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  after_previous();
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), kPairTmem);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist and the columns are held before any remote use
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  next_may_start();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // The issuing warps run whole (every lane waits, one elected lane issues), so that
    // loop counters, addresses and descriptors stay in the uniform datapath: with the
    // loops in one lane's branch a product took about 85 cycles to issue, and a k-block's
    // waits, products and commits more than its 512 cycles of tensor work
    if (warp == 0) {
      // ---------------- TMA producer (both CTAs: this CTA's halves)
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        int bm, bn;
        banded_tile(t, mt, nt, kBand, bm, bn);
        const int ma = bm * PM + 128 * rank, nb = bn * PN + 128 * rank;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = int(it % PSTAGES);
          ok = mbar_wait(empty_bar(s), ((it / PSTAGES) & 1u) ^ 1u, g.status, 31);
          if (!ok) break;
          const uint32_t a_dst = base + uint32_t(s) * PSTAGE_BYTES, b_dst = a_dst + HALF_STAGE;
          const uint32_t fb = map_rank(full_bar(s), 0);
          if (elect_one()) {
            if (rank == 0) mbar_expect_tx(full_bar(s), 2 * PSTAGE_BYTES);
            tma_load_2d_pair(a_dst, &tmX, kb * BK, ma, fb);
            if (TRANS)
              tma_load_2d_pair(b_dst, &tmW, nb, kb * BK, fb);
            else
              tma_load_2d_pair(b_dst, &tmW, kb * BK, nb, fb);
          }
          __syncwarp();
        }
      }
      // drain (leader): the pair's last copies have landed; the peer waits for this at
      // the closing cluster barrier
      if (rank == 0)
        for (uint32_t d = it > uint32_t(PSTAGES) ? it - PSTAGES : 0; d < it; ++d)
          mbar_wait(full_bar(int(d % PSTAGES)), (d / PSTAGES) & 1u, g.status, 32);
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (leader)
      const uint32_t id = idesc_e4m3(PM, PN, TRANS ? 1 : 0);
      const uint32_t total = uint32_t((ntiles - pair + npairs - 1) / npairs) * uint32_t(nk);
      uint32_t it = 0;
      bool ok = true;
      for (; it < total; ++it) {
        const int s = int(it % PSTAGES), buf = int(it & 1u);
        ok = mbar_wait(full_bar(s), (it / PSTAGES) & 1u, g.status, 34);
        if (!ok) break;
        const uint32_t a_addr = base + uint32_t(s) * PSTAGE_BYTES, b_addr = a_addr + HALF_STAGE;
        // K-major: rows 128 bytes apart, 32-code k slices 32 bytes apart; MN-major: a
        // column is a byte, 32 k rows of 128 bytes a slice
        const uint64_t ad = sdesc(a_addr, 16, 1024), bd = TRANS ? sdesc(b_addr, BK * 128, 1024) : sdesc(b_addr, 16, 1024);
        if (it >= 2) ok = mbar_wait_cluster_relaxed(tempty_bar(buf), ((it >> 1) & 1u) ^ 1u, g.status, 33);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_e4m3_pair(tmem + uint32_t(buf) * PN, ad + uint64_t(2 * kk), bd + uint64_t(TRANS ? 256 * kk : 2 * kk), id,
                          kk != 0 ? 1u : 0u);
          mma_commit_pair(tfull_bar(buf));
          mma_commit_pair(empty_bar(s));
        }
        __syncwarp();
      }
      // every product issued here has finished before the accumulators are freed
      if (it > 0 && ok) mbar_wait(tfull_bar(int((it - 1) & 1u)), ((it - 1) >> 1) & 1u, g.status, 36);
    } else if (warp == 2) {
      // ---------------- X's scales (both CTAs: this CTA's 128 rows)
      const uint32_t dst = base + OFF_SCALES + 16u * uint32_t(lane);
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        int bm, bn;
        banded_tile(t, mt, nt, kBand, bm, bn);
        const int row = bm * PM + 128 * rank + 4 * lane, bytes = 4 * max(0, min(4, g.n - row));
        const float* xs = g.xs + (bytes ? row : 0);  // (rows past the last read as 0)
        for (int kb = 0; kb < nk; ++kb, ++it, xs += g.ld_xs) {
          const int l = int(it % SLOTS);
          ok = mbar_wait(sempty_bar(l), ((it / SLOTS) & 1u) ^ 1u, g.status, 37);
          if (!ok) break;
          copy16_clipped(dst + uint32_t(l) * SLOT_BYTES, xs, bytes);
          copies_arrive(sfull_bar(l));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
    // ---------------- scaled accumulation and output (both CTAs: this CTA's 128 rows)
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t te0 = map_rank(tempty_bar(0), 0);
    const uint32_t box = base + OFF_OUT + uint32_t(warp - 4) * OUT_BOX;
    const uint32_t my_scale = base + OFF_SCALES + 4u * uint32_t(32 * q + lane);
    const uint32_t acc0 = tmem + (uint32_t(32 * q) << 16) + uint32_t(part) * PCOLS;
    const int64_t ws_step = TRANS ? g.tile_cols : 1;
    uint32_t it = 0;
    bool ok = true;
    for (int t = pair; ok && t < ntiles; t += npairs) {
      int bm, bn;
      banded_tile(t, mt, nt, kBand, bm, bn);
      const int row0 = bm * PM + 128 * rank + 32 * q;                        // the warp's first row of out
      const int c0 = bn * PN + PCOLS * part;                                 // its 64 columns
      const float* ws = TRANS ? g.ws + (c0 >> 7) : g.ws + int64_t(c0 >> 7) * g.tile_cols;
      float acc[PCOLS];
#pragma unroll
      for (int j = 0; j < PCOLS; ++j) acc[j] = 0.f;
      // W's scales for 32 k-blocks, block kb + l in lane l
      float wl = 0.f, wn = c0 < g.width && lane < nk ? __ldg(ws + lane * ws_step) : 0.f;
      for (int kb = 0; kb < nk; ++kb, ++it) {
        if ((kb & 31) == 0) {
          wl = wn;
          wn = c0 < g.width && kb + 32 + lane < nk ? __ldg(ws + int64_t(kb + 32 + lane) * ws_step) : 0.f;
        }
        const uint32_t buf = it & 1u, l = it % SLOTS;
        const float w = __shfl_sync(0xFFFFFFFFu, wl, kb & 31);
        ok = mbar_wait(sfull_bar(int(l)), (it / SLOTS) & 1u, g.status, 38);
        if (!ok) break;
        float f;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(my_scale + l * SLOT_BYTES) : "memory");
        f *= w;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(sempty_bar(int(l)));
        ok = mbar_wait(tfull_bar(int(buf)), (it >> 1) & 1u, g.status, 35);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < PCOLS; j += 32) {
          uint32_t r[32];
          tmem_ld32(acc0 + buf * PN + uint32_t(j), r);
          if (j + 32 == PCOLS) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(te0 + 8u * buf);
          }
          add_scaled<32>(acc + j, r, f);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last box has been read
        __syncwarp();
        put_box<32>(acc + 32 * u, box, lane);
        store_box<32>(g.out, g.ldo, g.n, g.width, g.bytes, &tmO, row0, c0 + 32 * u, box, lane);
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (the lanes that stored)
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmem);
  }
}

// ---------------------------------------------------------------- weight gradient
// dW = dY^T X in bf16 on the same pairs and tiles: both operands MN-major (a token's row
// holds 64-column chunks of 128 bytes), the summed index is the tokens, one accumulator of
// a tile's whole sum, two of them in turn.  The tile leaves as in k_linear_pair; a split
// product's fp32 sums leave from registers.  Bound by the products: 8192 tokens, 14336 x
// 4096 take 520 us with X's conversion to bf16 (15), 1.85 PFLOP/s, and 587 in a run of
// seconds under the power limit; a library's bf16 product of that size reaches 1.91 and 1.7.
// Few tokens are bound by the tiles' stores (64: 24 us for 117 MB of dW, 4.9 TB/s; with two
// stores of 64-byte rows a warp in place of one of whole lines 33).
constexpr int DK = 64;                          // tokens of a k-block
constexpr int CHUNK = DK * 128;                 // 64 tokens x 64 columns of bf16: 8 KB, two an operand
constexpr int DW_STAGES = 5, DW_BOX = 32 * 128;  // (a warp's staging of out: 32 rows x 64 bf16)
constexpr int DW_SMEM = 1024 + DW_STAGES * PSTAGE_BYTES + PEPI * DW_BOX;

struct DwKernelArgs {
  __nv_bfloat16* out;
  float* part;           // a split product's shares (k_dw_join), or NULL
  int64_t ldo, n;
  int rows, cols, splits;
  int chunk_boxes;       // dY's copies bring one chunk each, not two
  int accumulate, bytes;
  int* status;
};

// A share's values as the epilogue warps hold them: float4 j of lane l (columns 4j .. of its
// row) at 32 j + l of warp w's 512, so that every store is whole lines (by rows, 16 bytes a
// lane, the same stores took 4 us longer).
__device__ __forceinline__ int64_t share_at(int t, int rank, int w) {
  return ((int64_t(t) * 2 + rank) * PEPI + w) * 512;
}

// Instruction descriptor, kind::f16: D fp32, A and B bf16, both MN-major
constexpr uint32_t kDwIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | (uint32_t(PN >> 3) << 17) |
                              (uint32_t(PM >> 4) << 24);

__global__ void __launch_bounds__(PAIR_THREADS, 1)
    k_dw_pair(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ CUtensorMap tmO, const DwKernelArgs g) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  __shared__ __align__(8) uint64_t bars[2 * DW_STAGES + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(DW_STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * DW_STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * uint32_t(2 * DW_STAGES + 2 + b); };

  const int rank = int(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = (g.rows + PM - 1) / PM, nt = (g.cols + PN - 1) / PN, ntiles = mt * nt, total = ntiles * g.splits;
  const int nk = int((g.n + DK - 1) / DK);
  const int pair = int(blockIdx.x >> 1), npairs = int(gridDim.x >> 1);
  // tile t: share t / ntiles of the tokens' blocks [k0, k1)
  auto tile_of = [&](int t, int& bm, int& bn, int& sp, int& k0, int& k1) {
    sp = t / ntiles;
    banded_tile(t - sp * ntiles, mt, nt, kBand, bm, bn);
    k0 = int(int64_t(nk) * sp / g.splits);
    k1 = int(int64_t(nk) * (sp + 1) / g.splits);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < DW_STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the leader's expect_tx
      mbar_init(empty_bar(s), 1);  // the leader's commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * PEPI);  // the epilogue warps of both CTAs
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  after_previous();
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), kPairTmem);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist and the columns are held before any remote use
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  next_may_start();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs: this CTA's halves)
    uint32_t it = 0;
    bool ok = true;
    for (int t = pair; ok && t < total; t += npairs) {
      int bm, bn, sp, k0, k1;
      tile_of(t, bm, bn, sp, k0, k1);
      const int ma = bm * PM + 128 * rank, nb = bn * PN + 128 * rank;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(empty_bar(s), ((it / DW_STAGES) & 1u) ^ 1u, g.status, 41);
        if (!ok) break;
        const uint32_t a_dst = base + uint32_t(s) * PSTAGE_BYTES, b_dst = a_dst + HALF_STAGE;
        const uint32_t fb = map_rank(full_bar(s), 0);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full_bar(s), 2 * PSTAGE_BYTES);
          if (g.chunk_boxes) {
            tma_load_2d_pair(a_dst, &tmY, ma, kb * DK, fb);
            tma_load_2d_pair(a_dst + CHUNK, &tmY, ma + 64, kb * DK, fb);
          } else {
            tma_load_3d_pair(a_dst, &tmY, kb * DK, ma / 64, fb);
          }
          tma_load_3d_pair(b_dst, &tmX, kb * DK, nb / 64, fb);
        }
        __syncwarp();
      }
    }
    // drain (leader): the pair's last copies have landed; the peer waits for this at
    // the closing cluster barrier
    if (rank == 0)
      for (uint32_t d = it > uint32_t(DW_STAGES) ? it - DW_STAGES : 0; d < it; ++d)
        mbar_wait(full_bar(int(d % DW_STAGES)), (d / DW_STAGES) & 1u, g.status, 42);
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer (leader)
    uint32_t it = 0, tc = 0;
    bool ok = true;
    for (int t = pair; ok && t < total; t += npairs) {
      int bm, bn, sp, k0, k1;
      tile_of(t, bm, bn, sp, k0, k1);
      const int buf = int(tc & 1u);
      if (tc >= 2) ok = mbar_wait_cluster_relaxed(tempty_bar(buf), ((tc >> 1) & 1u) ^ 1u, g.status, 43);
      if (!ok) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(full_bar(s), (it / DW_STAGES) & 1u, g.status, 44);
        if (!ok) break;
        tc_fence_after();
        // 64-column chunks 8 KB apart, 16 tokens (2 KB) a product
        const uint64_t ad = sdesc(base + uint32_t(s) * PSTAGE_BYTES, CHUNK, 1024);
        const uint64_t bd = sdesc(base + uint32_t(s) * PSTAGE_BYTES + HALF_STAGE, CHUNK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_pair(tmem + uint32_t(buf) * PN, ad + uint64_t(128 * kk), bd + uint64_t(128 * kk), kDwIdesc,
                          kb != k0 || kk != 0 ? 1u : 0u);
          mma_commit_pair(empty_bar(s));
          if (kb + 1 == k1) mma_commit_pair(tfull_bar(buf));
        }
        __syncwarp();
      }
      if (ok) ++tc;
    }
    // every product issued here has finished before the accumulators are freed
    if (tc > 0 && ok) mbar_wait(tfull_bar(int((tc - 1) & 1u)), ((tc - 1) >> 1) & 1u, g.status, 46);
  } else if (warp >= 4) {
    // ---------------- output (both CTAs: this CTA's 128 rows)
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t te0 = map_rank(tempty_bar(0), 0);
    const uint32_t box = base + DW_STAGES * PSTAGE_BYTES + uint32_t(warp - 4) * DW_BOX;
    uint32_t tc = 0;
    for (int t = pair; t < total; t += npairs, ++tc) {
      int bm, bn, sp, k0, k1;
      tile_of(t, bm, bn, sp, k0, k1);
      const uint32_t buf = tc & 1u;
      if (!mbar_wait(tfull_bar(int(buf)), (tc >> 1) & 1u, g.status, 45)) break;
      tc_fence_after();
      const int row0 = bm * PM + 128 * rank + 32 * q, c0 = bn * PN + 64 * part;
      uint32_t r[64];
      const uint32_t at = tmem + (uint32_t(32 * q) << 16) + buf * PN + uint32_t(64 * part);
      tmem_ld32(at, r);
      tmem_ld32(at + 32, r + 32);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(te0 + 8u * buf);
      const int row = row0 + lane;
      if (g.part) {
        float4* o = reinterpret_cast<float4*>(g.part) + share_at(t, rank, warp - 4) + lane;
        if (row0 < g.rows && c0 < g.cols)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[32 * j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                    __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
        continue;
      }
      if (g.accumulate && row < g.rows) {
        const __nv_bfloat16* o = g.out + int64_t(row) * g.ldo + c0;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (c0 + j < g.cols) r[j] = __float_as_uint(__uint_as_float(r[j]) + __bfloat162float(o[j]));
      }
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last box has been read
      __syncwarp();
      put_box<64>(reinterpret_cast<const float*>(r), box, lane);
      store_box<64>(g.out, g.ldo, g.rows, g.cols, g.bytes, &tmO, row0, c0, box, lane);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (the lanes that stored)
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmem);
  }
}

// dw = sum of the shares in order (+ dw): a warp takes 32 rows x 16 columns
__global__ void __launch_bounds__(256) k_dw_join(const DwKernelArgs g) {
  after_previous();
  next_may_start();
  const int mt = (g.rows + PM - 1) / PM, nt = (g.cols + PN - 1) / PN, ntiles = mt * nt;
  const int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, h = int(i & 3), w = int(i >> 2) & (PEPI - 1), rank = int(i >> 6) & 1, t = int(i >> 7);
  int bm, bn;
  banded_tile(t, mt, nt, kBand, bm, bn);
  const int row = bm * PM + 128 * rank + 32 * (w & 3) + lane, c0 = bn * PN + 64 * (w >> 2) + 16 * h;
  if (row >= g.rows || c0 >= g.cols) return;
  const float4* p = reinterpret_cast<const float4*>(g.part) + share_at(t, rank, w) + 128 * h + lane;
  float4 v[4] = {};
  for (int k = 0; k < g.splits; ++k, p += share_at(ntiles, 0, 0))
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = p[32 * j];
      v[j].x += x.x, v[j].y += x.y, v[j].z += x.z, v[j].w += x.w;
    }
  const float* f = reinterpret_cast<const float*>(v);
  __nv_bfloat16* o = g.out + int64_t(row) * g.ldo + c0;  // (cols is a multiple of 16)
  alignas(16) __nv_bfloat16 y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = __float2bfloat16_rn(g.accumulate ? f[e] + __bfloat162float(o[e]) : f[e]);
  if (g.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0) {
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(y);
    *reinterpret_cast<uint4*>(o + 8) = *reinterpret_cast<const uint4*>(y + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = y[e];
  }
}

// X's scales at a pitch whose rows 16-byte copies can read
__global__ void __launch_bounds__(256) k_copy_scales(const float* __restrict__ x, int64_t ldx, int64_t n,
                                                     float* __restrict__ out, int64_t ldo) {
  after_previous();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) out[int64_t(blockIdx.y) * ldo + i] = x[int64_t(blockIdx.y) * ldx + i];
}

// k_linear's stages and dynamic shared memory for a_rows rows of X a stage.  The X stages come
// last, and a product reads 128 rows of the last one whatever it holds: what follows it is
// spare shared memory.
struct SmallPlan {
  int stages, smem;
};
constexpr SmallPlan small_plan(int a_rows) {
  const int stage = B_STAGE + a_rows * BK, spare = (BM - a_rows) * BK, part = BM * kPartPitch * 4;
  const int fit = (kSmem - 1024 - spare) / stage, stages = fit < kMaxStages ? fit : kMaxStages;
  const int bytes = stages * stage + spare;
  return {stages, 1024 + (part > bytes ? part : bytes)};
}

// The CTAs of a cluster wait for one another while they hold tensor memory, so a CTA must never
// wait for columns that a CTA of another cluster kernel holds on its SM (each cluster could
// hold what the other needs on another SM).  Shared memory sees to that: an SM holds two
// CTAs of k_linear (their columns fit) or one of a pair's, never both, and never one
// of either beside a pair of the Newton-Schulz products (which asserts the same).
constexpr bool small_ctas_are(int per_sm, int beside) {
  for (int rows = 8; rows <= BM; rows += 8)
    if (small_plan(rows).smem < kClusterSmemLeast || (per_sm + 1) * small_plan(rows).smem <= kSmemOfSm ||
        small_plan(rows).smem + beside <= kSmemOfSm)
      return false;
  return true;
}
static_assert(2 * kTmemCols <= 512 && small_ctas_are(2, PAIR_SMEM) && small_ctas_are(2, DW_SMEM), "k_linear's CTAs");
static_assert(2 * PAIR_SMEM > kSmemOfSm && 2 * DW_SMEM > kSmemOfSm && PAIR_SMEM + DW_SMEM > kSmemOfSm, "the pairs' CTAs");
static_assert(PAIR_SMEM >= kClusterSmemLeast && DW_SMEM >= kClusterSmemLeast, "beside the Newton-Schulz pairs");

// slots[k]: clusters of k CTAs that fit the device at once with an SM for each CTA
// (k_linear_pair's shared memory sees to that), k = 1 .. 8: 152 SMs hold 76 of two, 46 of
// three, 36 of four, 15 of eight.  Found once per device; the SMs' share where the occupancy
// query fails.
const int* cluster_slots() {
  static std::mutex mu;
  static int cached[65][9] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 64;
  std::lock_guard<std::mutex> lock(mu);
  int* slots = cached[dev];
  if (slots[1] == 0) {
    const int sms = sm_count();
    cudaFuncSetAttribute(k_linear_pair<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, PAIR_SMEM);
    for (int size = 2; size <= 8; ++size) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = unsigned(size);
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(unsigned(size * sms));
      cfg.blockDim = dim3(PAIR_THREADS);
      cfg.dynamicSmemBytes = PAIR_SMEM;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&slots[size], k_linear_pair<false>, &cfg) != cudaSuccess || slots[size] < 1) {
        cudaGetLastError();
        slots[size] = sms / size;
      }
    }
    slots[1] = sms;
  }
  return slots;
}

int launch_clusters(const void* kernel, int clusters, int size, int threads, int smem, void** args, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(size);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (after_previous)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(clusters) * unsigned(size));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaLaunchKernelExC(&cfg, kernel, args);
  return check("bq_linear_fp8");
}

}  // namespace

int launch_linear_fp8(const LinearArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static OncePerDevice once;
  if (int rc = once.run(current_device(), [] {
        if (cudaFuncSetAttribute(k_linear<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(k_linear<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(k_linear_pair<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, PAIR_SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(k_linear_pair<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, PAIR_SMEM) != cudaSuccess)
          return check("bq_linear_fp8 (shared memory attribute)");
        return int(BQ_OK);
      }))
    return rc;
  const int width = a.transposed ? a.cols : a.rows, red = a.transposed ? a.rows : a.cols;
  LinArgs g;
  g.xs = a.x_scale, g.ws = a.w_scale, g.out = static_cast<__nv_bfloat16*>(a.out);
  g.ld_xs = a.ld_xs, g.ldo = a.ldo, g.n = int(a.n), g.width = width, g.red = red;
  g.tile_cols = (a.cols + 127) / 128, g.status = a.status;
  g.split = 1, g.stages = 0, g.a_rows = BM, g.bytes = store_bytes(a.out, a.ldo, width);
  const int nk = (red + BK - 1) / BK;
  CUtensorMap tx, tw, to;
  if (int rc = encode_map_codes(&tw, a.w, a.cols, a.rows, a.ldw, 128)) return rc;
  const int64_t pairs = ((a.n + PM - 1) / PM) * ((width + PN - 1) / PN);
  const int64_t tiles = ((a.n + BM - 1) / BM) * ((width + BN - 1) / BN);
  if (tiles > 0x7FFFFFF) return set_error(BQ_EINVAL, "bq_linear_fp8: too many tiles");
  // k_linear: into how many CTAs to split a tile's k-blocks, by the times of 30 products.  A
  // CTA alone on its SM takes 0.35 us a k-block (transposed 0.40), two on one 0.4 to 0.6 each, and a
  // join by rows and shares; not into a second wave (75 tiles of 16 k-blocks: 8.5 us by 2, 14.9
  // by 4).  128 rows and more, 48 tiles of 16: 8.2 us by 2, 10.1 by 4; 50 of 105: 23.6 by 2, 28.2
  // by 3, 26.8 by 4; 100 of 64: 27.9 in one, 20.7 by 2; one row, 64 tiles of 64: 15.1 by 2,
  // 13.7 by 4.
  const int* slots = cluster_slots();
  const int64_t waves = (tiles + 2 * slots[1] - 1) / (2 * slots[1]);
  const double one = a.transposed ? 0.40 : 0.35, full = double(std::min<int64_t>(a.n, BM)) / BM;
  double us_one = tiles <= slots[1] ? 5 + one * nk : 2 + double(waves) * (6 + 0.52 * nk);
  for (int k = 2; k <= 8 && k <= nk && tiles <= 2 * slots[k]; ++k) {
    const int share = (nk + k - 1) / k;
    const double us = tiles <= slots[k] ? 5 + one * share + (k - 1) * (0.12 + 0.2 * full)
                                        : 6 + (k == 2 ? 0.4 + 0.1 * full : 0.45 + 0.15 * full) * share + (k - 1) * (0.25 + 0.55 * full);
    if (us < us_one) us_one = us, g.split = k;
  }
  // The pairs take more than 128 rows (fewer leave one of the CTAs idle: 12 rows of 11048 x
  // 5952 take 28 us there and 17 us on k_linear), where their tiles take less time: 0.40 us a k-block
  // and 2.5 us a wave.  337 rows of 11840 x 4512 (two waves, or one of k_linear's): 38.3 us on
  // pairs, 25.5 on k_linear; 849 of 6336 x 8144 (two and two): 64.2 and 96.1; 512 of 8192 x
  // 4096 (one and one): 18.5 and 24.2.
  const double us_pair = 4 + double((pairs + slots[2] - 1) / slots[2]) * (0.40 * nk + 2.5);
  if (a.n > BM && us_pair < us_one) {
    if (int rc = encode_map_codes(&tx, a.x, red, a.n, a.ldx, 128)) return rc;
    to = tx;  // (not read by plain stores)
    if (a.ld_xs % 4 || (reinterpret_cast<uintptr_t>(a.x_scale) & 15)) {
      const int64_t ld = (a.n + 3) / 4 * 4;
      k_copy_scales<<<dim3(unsigned((a.n + 255) / 256), unsigned(nk)), 256, 0, s>>>(a.x_scale, a.ld_xs, a.n, a.scale_ws, ld);
      if (int rc = check("bq_linear_fp8 (scales)")) return rc;
      g.xs = a.scale_ws, g.ld_xs = ld;
    }
    if (g.bytes == 16)
      if (int rc = encode_map_bf16_out(&to, a.out, width, a.n, a.ldo, 32)) return rc;
    void* args[] = {&tx, &tw, &to, &g};
    const void* k = a.transposed ? reinterpret_cast<const void*>(k_linear_pair<true>)
                                 : reinterpret_cast<const void*>(k_linear_pair<false>);
    return launch_clusters(k, int(std::min<int64_t>(pairs, slots[2])), 2, PAIR_THREADS, PAIR_SMEM, args, s);
  }
  g.a_rows = int(std::min<int64_t>(BM, (a.n + 7) / 8 * 8));
  const SmallPlan plan = small_plan(g.a_rows);
  g.stages = plan.stages;
  if (int rc = encode_map_codes(&tx, a.x, red, a.n, a.ldx, g.a_rows)) return rc;
  void* args[] = {&tx, &tw, &g};
  const void* k = a.transposed ? reinterpret_cast<const void*>(k_linear<true>) : reinterpret_cast<const void*>(k_linear<false>);
  return launch_clusters(k, int(tiles), g.split, THREADS, plan.smem, args, s);
}

size_t dw_part_bytes(int splits, int64_t rows, int64_t cols) {
  return splits > 1 ? size_t(splits) * size_t((rows + PM - 1) / PM) * size_t((cols + PN - 1) / PN) * PM * PN * 4 : 0;
}

// A product of few tiles and many tokens leaves most pairs idle: its tokens are split where
// that costs less, by the times of 1, 6 and 16 tiles: 0.29 us a k-block, and for shares a
// launch, their stores and their sums.  1024 x 1024: 1000 tokens 11.4 us in one, 13.2 in two
// and 15.0 in four shares; 8000 tokens 43.7, 31.9 and 27.4.
int dw_splits(int64_t n, int64_t rows, int64_t cols) {
  const int64_t tiles = ((rows + PM - 1) / PM) * ((cols + PN - 1) / PN), nk = (n + DK - 1) / DK;
  const int most = int(std::min<int64_t>({sm_count() / 2 / tiles, nk, 16}));
  int best = 1;
  double least = 0.29 * double(nk);
  for (int s = 2; s <= most; ++s) {
    const double us = 0.29 * double((nk + s - 1) / s) + 2.2 + s * (0.25 + 0.045 * double(tiles));
    if (us < least) least = us, best = s;
  }
  return best;
}

int launch_dw(const DwArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static OncePerDevice once;
  if (int rc = once.run(current_device(), [] {
        if (cudaFuncSetAttribute(k_dw_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, DW_SMEM) != cudaSuccess)
          return check("bq_linear_fp8_dw (shared memory attribute)");
        return int(BQ_OK);
      }))
    return rc;
  DwKernelArgs g;
  g.out = static_cast<__nv_bfloat16*>(a.dw);
  g.ldo = a.ld_dw, g.n = a.n, g.rows = a.rows, g.cols = a.cols, g.status = a.status;
  g.splits = dw_splits(a.n, a.rows, a.cols);
  g.part = g.splits > 1 ? a.part : nullptr;
  g.chunk_boxes = a.padded ? 0 : 1;
  g.accumulate = a.accumulate;
  g.bytes = store_bytes(a.dw, a.ld_dw, a.cols);
  CUtensorMap ty, tx, to;
  if (int rc = encode_map_chunks(&ty, a.dy, a.rows, a.n, a.ld_dy, a.padded ? 2 : 0)) return rc;
  if (int rc = encode_map_chunks(&tx, a.x, a.cols, a.n, a.ld_x, 2)) return rc;
  to = tx;  // (not read by plain stores)
  if (g.bytes == 16)
    if (int rc = encode_map_bf16_out(&to, a.dw, a.cols, a.rows, a.ld_dw, 64)) return rc;
  const int64_t tiles = int64_t((a.rows + PM - 1) / PM) * ((a.cols + PN - 1) / PN) * g.splits;
  void* args[] = {&ty, &tx, &to, &g};
  if (int rc = launch_clusters(reinterpret_cast<const void*>(k_dw_pair), int(std::min<int64_t>(tiles, cluster_slots()[2])), 2,
                               PAIR_THREADS, DW_SMEM, args, s))
    return rc;
  if (!g.part) return BQ_OK;
  launch_after(k_dw_join, unsigned(tiles / g.splits * 16), 256, 0, s, g);
  return check("bq_linear_fp8_dw (join)");
}

}  // namespace bq
