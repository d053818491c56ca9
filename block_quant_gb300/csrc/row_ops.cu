// Row-wise operators of a layer around the DBuffer step on GB300 (sm_103a):
//   k_embed          rows of the token table (bf16, or E4M3 codes with 128x128
//                    tile scales as the AllGather leaves them) times a factor
//   k_embed_sort     stable sort of a batch's tokens by id (one cluster)
//   k_embed_pieces,  the table's gradient: rows of dY summed over equal ids
//   k_embed_rows
//   k_norm*          residual addition, root-mean-square norm, E4M3 codes with
//                    one scale per 128 values of a row (also without the norm:
//                    the row quantiser)
//   k_norm_grad*     the norm's gradients
// All are bound by memory: each reads its inputs once and writes its outputs once.
#include <algorithm>
#include <string>

#include "bq_internal.h"
#include "fp8_codes.h"
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

template <bool VEC, bool FP8>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_embed(const void* __restrict__ table, const float* __restrict__ tscale, int64_t rows, int cols, int64_t ldt,
            const void* __restrict__ ids, int id_bits, int64_t n, float scale, __nv_bfloat16* __restrict__ out,
            int64_t ldo, int segs) {
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
#pragma unroll
      for (int j = 0; j < kSpans; ++j) {
        if (VEC) {
          const int c = c0 + kSpan * j + 8 * lane;
          if (c >= cols) continue;
          decode8(__ldg(reinterpret_cast<const uint2*>(row + c)), v[j]);
          const float s = __ldg(srow + (c >> 7));
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = __fmul_rn(v[j][e], s);
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

// A stable least-significant-digit radix sort of (id, position) in one launch: a
// cluster of eight CTAs, each owning a contiguous eighth of the tokens.  Per
// digit: CTA histograms, exchanged through distributed shared memory and scanned
// by every CTA; then ranks in token order, 1024 x kSortKeys tokens a round, by
// warp match and per-warp counters; the pairs go to the other buffer, which the
// cluster barrier makes visible.  Ids outside [0, rows) become `rows` (last).
constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = 32, kSortKeys = 4;
constexpr int kDigit = 9, kBins = 1 << kDigit;

struct SortSmem {
  uint32_t hist[kBins];              // this CTA's count of every digit (read by the whole cluster)
  uint32_t base[kBins];              // where this CTA's next token of a digit goes
  uint32_t round[kBins];             // a round's count of every digit
  uint32_t warp_sum[kSortWarps];
  uint16_t count[kSortWarps][kBins];  // a round's counts, then offsets, by warp
};

__global__ void __launch_bounds__(kSortThreads, 1) __cluster_dims__(kSortCtas, 1, 1)
    k_embed_sort(const void* __restrict__ ids, int id_bits, int n, int rows, int passes, uint2* __restrict__ buf0,
                 uint2* __restrict__ buf1) {
  __shared__ SortSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = int(cluster_rank());
  const int seg = (n + kSortCtas - 1) / kSortCtas;
  const int lo = min(n, rank * seg), hi = min(n, lo + seg);
  for (int p = 0; p < passes; ++p) {
    const uint2* src = (p & 1) ? buf1 : buf0;  // pass 0 reads the ids themselves
    uint2* dst = (p & 1) ? buf0 : buf1;
    const int shift = p * kDigit;
    auto key_at = [&](int i) -> uint2 {
      if (p > 0) return __ldcg(src + i);
      const int64_t id = load_id(ids, id_bits, i);
      return make_uint2(id >= 0 && id < rows ? uint32_t(id) : uint32_t(rows), uint32_t(i));
    };
    if (tid < kBins) sm.hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kSortThreads) atomicAdd(&sm.hist[(key_at(i).x >> shift) & (kBins - 1)], 1u);
    cluster_sync();
    // exclusive scan over (digit, CTA): thread d < kBins holds digit d
    uint32_t before = 0, total = 0;
    if (tid < kBins) {
      const uint32_t at = smem_addr(&sm.hist[tid]);
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        uint32_t h;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(h) : "r"(map_rank(at, uint32_t(c))) : "memory");
        if (c < rank) before += h;
        total += h;
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
      uint32_t prior = 0;
      for (int w = 0; w < warp; ++w) prior += sm.warp_sum[w];
      sm.base[tid] = prior + x - total + before;
    }
    // ranks, in token order
    for (int r0 = lo; r0 < hi; r0 += kSortThreads * kSortKeys) {
      for (int i = tid; i < kSortWarps * kBins / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(sm.count)[i] = 0;
      __syncthreads();
      uint2 kv[kSortKeys];
      uint32_t off[kSortKeys];
      const int w0 = r0 + warp * 32 * kSortKeys;
#pragma unroll
      for (int j = 0; j < kSortKeys; ++j) {
        const int i = w0 + 32 * j + lane;
        if (i < hi) kv[j] = key_at(i);
      }
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
      if (tid < kBins) {  // counts -> offsets of each warp inside the round
        uint32_t run = 0;
        for (int w = 0; w < kSortWarps; ++w) {
          const uint32_t c = sm.count[w][tid];
          sm.count[w][tid] = uint16_t(run);
          run += c;
        }
        sm.round[tid] = run;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSortKeys; ++j) {
        if (w0 + 32 * j + lane >= hi) continue;
        const uint32_t d = (kv[j].x >> shift) & (kBins - 1);
        dst[sm.base[d] + sm.count[warp][d] + off[j]] = kv[j];
      }
      __syncthreads();
      if (tid < kBins) sm.base[tid] += sm.round[tid];
    }
    __threadfence();
    cluster_sync();  // the next pass reads other CTAs' pairs; their histograms are done being read
  }
}

// ---------------------------------------------------------------- embedding gradient

// dT[v] (+)= f * sum of dY[t] over the tokens t of id v, summed in fp32 in token
// order.  The sorted tokens are cut into pieces of kPiece: a run of equal ids
// inside one piece is summed where its row is written (k_embed_rows); a run that
// crosses a piece's end is summed piece by piece first (k_embed_pieces), so a
// token that fills the batch is shared out over the whole GPU, and its row adds
// the pieces' sums in order.  No atomics: the same batch gives the same bits.
// Sum slot of a piece: 2c if its run begins at or before piece c's first token,
// 2c + 1 if it begins inside.
constexpr int kPiece = 32;

// sum of rows dY[pos[i]] over i in [b, e), one span
template <bool VEC>
__device__ __forceinline__ void sum_rows(const __nv_bfloat16* __restrict__ dy, int64_t ld, const uint32_t* pos, int b,
                                         int e, int c0, int cols, int lane, float* acc) {
  int i = b;
  for (; i + 4 <= e; i += 4) {
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) load_bf16<VEC>(dy + int64_t(pos[i + k]) * ld, c0, cols, lane, v[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[k][x]);
  }
  for (; i < e; ++i) {
    float v[8];
    load_bf16<VEC>(dy + int64_t(pos[i]) * ld, c0, cols, lane, v);
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[x]);
  }
}

// blockIdx.x: piece; blockIdx.y: group of kPieceWarps spans
constexpr int kPieceWarps = 4;
template <bool VEC>
__global__ void __launch_bounds__(32 * kPieceWarps)
    k_embed_pieces(const uint2* __restrict__ sorted, int n, int rows, const __nv_bfloat16* __restrict__ dy, int64_t ld,
                   int cols, float* __restrict__ sums, int ldp) {
  __shared__ uint32_t key[kPiece + 2], pos[kPiece];  // key[1 + i]: token i of the piece; 0, len + 1: its neighbours
  const int b = blockIdx.x * kPiece, len = min(kPiece, n - b);
  const int tid = threadIdx.x;
  if (tid < len + 2) {
    const int i = b + tid - 1;
    const uint2 kv = i >= 0 && i < n ? sorted[i] : make_uint2(0xFFFFFFFFu, 0u);
    key[tid] = kv.x;
    if (tid >= 1 && tid <= len) pos[tid - 1] = kv.y;
  }
  __syncthreads();
  const uint32_t first = key[1], last = key[len];
  const bool from = key[0] == first, to = key[len + 1] == last;
  const int lane = tid & 31, c0 = (int(blockIdx.y) * kPieceWarps + (tid >> 5)) * kSpan;
  if (c0 >= cols) return;
  int head = 0, tail = len;  // [0, head) and [tail, len) are pieces of runs that cross the ends
  if (from || (to && first == last)) {
    while (head < len && key[1 + head] == first) ++head;
  }
  if (to && head < len) {
    while (tail > head && key[tail] == last) --tail;
  }
  if (head > 0 && first < uint32_t(rows)) {
    float acc[8] = {};
    sum_rows<VEC>(dy, ld, pos, 0, head, c0, cols, lane, acc);
    store_f32<true>(sums + int64_t(2 * blockIdx.x) * ldp, c0, ldp, lane, acc);
  }
  if (tail < len && last < uint32_t(rows)) {
    float acc[8] = {};
    sum_rows<VEC>(dy, ld, pos, tail, len, c0, cols, lane, acc);
    store_f32<true>(sums + int64_t(2 * blockIdx.x + 1) * ldp, c0, ldp, lane, acc);
  }
}

// a CTA writes kTableRows rows of the table's gradient
constexpr int kTableRows = 64;
template <bool VEC, typename Out>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_embed_rows(const uint2* __restrict__ sorted, int n, int64_t rows, const __nv_bfloat16* __restrict__ dy,
                 int64_t ld, int cols, const float* __restrict__ sums, int ldp, float scale, int accumulate,
                 Out* __restrict__ out, int64_t ldo) {
  __shared__ int first[kTableRows + 1];  // first sorted token of each row
  __shared__ uint32_t pos[kRowWarps][kPiece];
  const int64_t v0 = int64_t(blockIdx.x) * kTableRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid <= kTableRows) {
    const uint32_t v = uint32_t(min(v0 + tid, rows));
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid].x < v)
        lo = mid + 1;
      else
        hi = mid;
    }
    first[tid] = lo;
  }
  __syncthreads();
  const int spans = (cols + kSpan - 1) / kSpan;
  const int count = int(min(int64_t(kTableRows), rows - v0));
  for (int item = warp; item < count * spans; item += kRowWarps) {
    const int r = item / spans, c0 = (item - r * spans) * kSpan;
    const int b = first[r], e = first[r + 1];
    if (b == e && accumulate) continue;
    float acc[8] = {};
    if (b < e) {
      const int p0 = b / kPiece, p1 = (e - 1) / kPiece;
      if (p0 == p1) {
        __syncwarp();
        if (lane < e - b) pos[warp][lane] = sorted[b + lane].y;
        __syncwarp();
        sum_rows<VEC>(dy, ld, pos[warp], 0, e - b, c0, cols, lane, acc);
      } else {
        for (int p = p0; p <= p1; ++p) {
          const int slot = p == p0 && b % kPiece != 0 ? 2 * p + 1 : 2 * p;
          float v[8];
          load_f32<true>(sums + int64_t(slot) * ldp, c0, ldp, lane, v);
          // the sums' rows hold whole spans: lane l has columns 8l .. 8l + 7 of
          // the span, or what column() gives where the span was summed unaligned
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[x] = __fadd_rn(acc[x], v[x]);
        }
      }
    }
    Out* row = out + (v0 + r) * ldo;
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
      for (int e = 0; e < 8; ++e) h[i][e] = __bfloat162float(__float2bfloat16_rn(h[i][e] + r[e]));
      if (a.h) store_bf16<VEC>(a.h + t * a.ldh, c0, a.cols, lane, h[i]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  ss = warp_sum(ss);
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

template <bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps)
    k_quant_rows(const __nv_bfloat16* __restrict__ x, int64_t ldx, int64_t n, int cols, uint8_t* __restrict__ codes,
                 int64_t ldc, float* __restrict__ scale, int64_t lds, int spans) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / spans;
  if (t >= n) return;
  const int c0 = int(item - t * spans) * kSpan;
  float v[8];
  load_bf16<VEC>(x + t * ldx, c0, cols, lane, v);
  quant_span<VEC>(v, c0, cols, lane, codes + t * ldc, scale + t, lds);
}

// bf16(scale * code) of E4M3 rows with one scale per 128 values, pitch ldo (for the
// weight gradient's product); cols is a multiple of 16, so every vector is aligned
__global__ void __launch_bounds__(32 * kRowWarps)
    k_dequant_rows(const uint8_t* __restrict__ codes, int64_t ldc, const float* __restrict__ scale, int64_t lds,
                   int64_t n, int cols, __nv_bfloat16* __restrict__ out, int64_t ldo, int spans) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / spans;
  if (t >= n) return;
  const int c = int(item - t * spans) * kSpan + 8 * lane;
  if (c >= cols) return;
  float v[8];
  decode8(__ldg(reinterpret_cast<const uint2*>(codes + t * ldc + c)), v);
  const float s = __ldg(scale + int64_t(c >> 7) * lds + t);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], s);
  *reinterpret_cast<uint4*>(out + t * ldo + c) = pack8(v);
}

// bf16 rows copied to a pitch of their own
__global__ void __launch_bounds__(32 * kRowWarps)
    k_copy_rows(const __nv_bfloat16* __restrict__ x, int64_t ldx, int64_t n, int cols, __nv_bfloat16* __restrict__ out,
                int64_t ldo, int spans) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / spans;
  if (t >= n) return;
  const int c0 = int(item - t * spans) * kSpan;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = c0 + 32 * e + lane;
    if (c < cols) out[t * ldo + c] = x[t * ldx + c];
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
__global__ void __launch_bounds__(row_threads(VPT)) k_norm_grad(const NormGradArgs a) {
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

// dw = sum of the CTAs' parts in order: 32 columns x 8 runs of parts a CTA
template <typename Out>
__global__ void __launch_bounds__(256)
    k_norm_dw(const float* __restrict__ part, int parts, int ldp, int cols, int accumulate, Out* __restrict__ dw) {
  __shared__ float run[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
    const int per = (parts + 7) / 8, b = warp * per, e = min(parts, b + per);
#pragma unroll 8
    for (int p = b; p < e; ++p) s += part[int64_t(p) * ldp + c];
  }
  run[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += run[k][lane];
    if (sizeof(Out) == 2) {
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(dw);
      if (accumulate) s += __bfloat162float(o[c]);
      o[c] = __float2bfloat16_rn(s);
    } else {
      float* o = reinterpret_cast<float*>(dw);
      if (accumulate) s += o[c];
      o[c] = s;
    }
  }
}

// ---------------------------------------------------------------- host

bool vec_ok(const void* p, int64_t ld, int values) { return aligned16(p) && ld % values == 0; }

// warps of a one-CTA-per-row kernel and spans a warp, within row_threads(spans a
// warp) threads for rows of up to 65536 columns
void row_shape(int cols, int* warps, int* vpt) {
  const int spans = (cols + kSpan - 1) / kSpan;
  *vpt = spans <= 32 ? 2 : spans <= 64 ? 4 : 8;
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
  p.pieces = int((n + kPiece - 1) / kPiece);
  p.off_b0 = 0;
  p.off_b1 = up(size_t(n) * 8);
  p.off_sums = p.off_b1 + up(size_t(n) * 8);
  p.bytes = p.off_sums + up(size_t(p.pieces) * 2 * size_t(p.ldp) * 4);
  if (p.bytes == 0) p.bytes = 256;
  return p;
}

int norm_grad_ctas(int64_t n) { return int(std::min<int64_t>(n, int64_t(sm_count()) * 2)); }

}  // namespace

int launch_embed(const EmbedArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = a.kind == BQ_ROWS_FP8;
  const bool vec = a.cols % 8 == 0 && vec_ok(a.out, a.ldo, 8) &&
                   (fp8 ? (reinterpret_cast<uintptr_t>(a.table) & 7) == 0 && a.ldt % 8 == 0 : vec_ok(a.table, a.ldt, 8));
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const int64_t ctas = (a.n * segs + kRowWarps - 1) / kRowWarps;
  auto* k = fp8 ? (vec ? k_embed<true, true> : k_embed<false, true>) : (vec ? k_embed<true, false> : k_embed<false, false>);
  k<<<unsigned(ctas), 32 * kRowWarps, 0, s>>>(a.table, a.tscale, a.rows, a.cols, a.ldt, a.ids, a.id_bits, a.n, a.scale,
                                              static_cast<__nv_bfloat16*>(a.out), a.ldo, segs);
  return check("bq_embed");
}

size_t embed_grad_bytes(int64_t n, int64_t cols) { return embed_grad_plan(n, cols).bytes; }

int launch_embed_grad(const EmbedGradArgs& a, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const EmbedGradPlan p = embed_grad_plan(a.n, a.cols);
  auto* w = static_cast<unsigned char*>(ws);
  auto* b0 = reinterpret_cast<uint2*>(w + p.off_b0);
  auto* b1 = reinterpret_cast<uint2*>(w + p.off_b1);
  auto* sums = reinterpret_cast<float*>(w + p.off_sums);
  const auto* dy = static_cast<const __nv_bfloat16*>(a.dy);
  const int n = int(a.n);
  const bool f32 = a.out_kind == BQ_ROWS_FP32;
  const bool vec = a.cols % 8 == 0 && vec_ok(a.dy, a.ld_dy, 8) && vec_ok(a.out, a.ldo, f32 ? 4 : 8);
  const int passes = (bits_of(a.rows) + kDigit - 1) / kDigit;
  const uint2* sorted = (passes & 1) ? b1 : b0;
  if (n > 0) {
    k_embed_sort<<<kSortCtas, kSortThreads, 0, s>>>(a.ids, a.id_bits, n, int(a.rows), passes, b0, b1);
    if (int rc = check("bq_embed_grad (sort)")) return rc;
    const dim3 g(unsigned(p.pieces), unsigned((a.cols + kPieceWarps * kSpan - 1) / (kPieceWarps * kSpan)));
    auto* kp = vec ? k_embed_pieces<true> : k_embed_pieces<false>;
    kp<<<g, 32 * kPieceWarps, 0, s>>>(sorted, n, int(a.rows), dy, a.ld_dy, a.cols, sums, p.ldp);
    if (int rc = check("bq_embed_grad (pieces)")) return rc;
  }
  const unsigned ctas = unsigned((a.rows + kTableRows - 1) / kTableRows);
  if (f32) {
    auto* k = vec ? k_embed_rows<true, float> : k_embed_rows<false, float>;
    k<<<ctas, 32 * kRowWarps, 0, s>>>(sorted, n, a.rows, dy, a.ld_dy, a.cols, sums, p.ldp, a.scale, a.accumulate,
                                      static_cast<float*>(a.out), a.ldo);
  } else {
    auto* k = vec ? k_embed_rows<true, __nv_bfloat16> : k_embed_rows<false, __nv_bfloat16>;
    k<<<ctas, 32 * kRowWarps, 0, s>>>(sorted, n, a.rows, dy, a.ld_dy, a.cols, sums, p.ldp, a.scale, a.accumulate,
                                      static_cast<__nv_bfloat16*>(a.out), a.ldo);
  }
  return check("bq_embed_grad (rows)");
}

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
  row_shape(r.cols, &warps, &vpt);
  auto* k = vec ? (vpt == 2 ? k_norm<true, 2> : vpt == 4 ? k_norm<true, 4> : k_norm<true, 8>)
                : (vpt == 2 ? k_norm<false, 2> : vpt == 4 ? k_norm<false, 4> : k_norm<false, 8>);
  k<<<unsigned(r.n), 32 * warps, 0, s>>>(a);
  return check("bq_rmsnorm");
}

int launch_quant_rows(const void* x, int64_t ldx, int64_t n, int cols, uint8_t* codes, int64_t ldc, float* scale,
                      int64_t lds, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = cols % 8 == 0 && vec_ok(x, ldx, 8) && (reinterpret_cast<uintptr_t>(codes) & 7) == 0 && ldc % 8 == 0;
  const int spans = (cols + kSpan - 1) / kSpan;
  const int64_t ctas = (n * spans + kRowWarps - 1) / kRowWarps;
  auto* k = vec ? k_quant_rows<true> : k_quant_rows<false>;
  k<<<unsigned(ctas), 32 * kRowWarps, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx, n, cols, codes, ldc, scale, lds,
                                              spans);
  return check("bq_quant_rows_fp8");
}

int launch_dequant_rows(const uint8_t* codes, int64_t ldc, const float* scale, int64_t lds, int64_t n, int cols,
                        void* out, int64_t ldo, void* stream) {
  const int spans = (cols + kSpan - 1) / kSpan;
  const int64_t ctas = (n * spans + kRowWarps - 1) / kRowWarps;
  k_dequant_rows<<<unsigned(ctas), 32 * kRowWarps, 0, static_cast<cudaStream_t>(stream)>>>(
      codes, ldc, scale, lds, n, cols, static_cast<__nv_bfloat16*>(out), ldo, spans);
  return check("bq_linear_fp8_dw (input)");
}

int launch_copy_rows(const void* x, int64_t ldx, int64_t n, int cols, void* out, int64_t ldo, void* stream) {
  const int spans = (cols + kSpan - 1) / kSpan;
  const int64_t ctas = (n * spans + kRowWarps - 1) / kRowWarps;
  k_copy_rows<<<unsigned(ctas), 32 * kRowWarps, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(x), ldx, n, cols, static_cast<__nv_bfloat16*>(out), ldo, spans);
  return check("bq_linear_fp8_dw (copy)");
}

size_t rmsnorm_grad_bytes(int64_t n, int64_t cols) {
  const size_t ldp = size_t((cols + kSpan - 1) / kSpan * kSpan);
  return std::max<size_t>(256, size_t(norm_grad_ctas(n)) * ldp * 4);
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
  const int ctas = norm_grad_ctas(r.n);
  if (ctas > 0) {
    const bool vec = r.cols % 8 == 0 && vec_ok(r.dy, r.ld_dy, 8) && vec_ok(r.h, r.ld_h, 8) && aligned16(r.weight) &&
                     (!r.dh || vec_ok(r.dh, r.ld_dh, 8)) && vec_ok(r.dx, r.ld_dx, 8);
    int warps, vpt;
    row_shape(r.cols, &warps, &vpt);
    auto* k = vec ? (vpt == 2 ? k_norm_grad<true, 2> : vpt == 4 ? k_norm_grad<true, 4> : k_norm_grad<true, 8>)
                  : (vpt == 2 ? k_norm_grad<false, 2> : vpt == 4 ? k_norm_grad<false, 4> : k_norm_grad<false, 8>);
    k<<<unsigned(ctas), 32 * warps, 0, s>>>(a);
    if (int rc = check("bq_rmsnorm_grad")) return rc;
  }
  const unsigned g = unsigned((r.cols + 31) / 32);
  if (r.dw_kind == BQ_ROWS_FP32)
    k_norm_dw<<<g, 256, 0, s>>>(a.part, ctas, a.ldp, r.cols, r.accumulate, static_cast<float*>(r.dw));
  else
    k_norm_dw<<<g, 256, 0, s>>>(a.part, ctas, a.ldp, r.cols, r.accumulate, static_cast<__nv_bfloat16*>(r.dw));
  return check("bq_rmsnorm_grad (dw)");
}

}  // namespace bq
