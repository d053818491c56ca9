// Softmax losses over an FP8 head (sm_103a): cross entropy of a class, and the divergence from
// a teacher's top logits, with their gradients.  With z = scale * X W^T (n tokens, a vocabulary
// of `rows`) and a row's targets q (weights of a few ids, of sum 1):
//   loss = sum_i q_i (log q_i - log p_i),  p = softmax(z),
//   dX = diag(g) scale U W,  dW = (diag(g) U)^T scale X,  U = p - q.
// z is never kept.  Forward: every tile of logits leaves the product (linear_fp8.cu) as its rows'
// statistics (loss_tile.h), which one launch joins.  Gradient: pieces of the vocabulary, one
// after another; a piece's logits are made again and leave as U in fp16, which two
// products read, with the piece of W for dX and with X for that piece of dW.
//
// fp16 and not bf16 or E4M3: U is in [-1, 1] and W and g X are brought to a common power of two
// first, so all three keep eleven bits over the top 28 powers of two, at the rate of bf16 products;
// what the results lose is their own rounding to bf16.  (E4M3 rows of U would make dX
// half as expensive and 2.5 % wrong.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <string>

#include "bq_internal.h"
#include "loss_tile.h"
#include "once.h"
#include "pair_tiles.h"
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

constexpr int kMaxPairs = 1024;  // of a row

__device__ __forceinline__ void decode16(const uint4& w, float* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {  // (NaN are passed over)
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// a row's targets
struct Targets {
  const void *ids, *teacher;
  int64_t ld_ids, ld_teacher;
  float scale;
  int rows, k, id_bits, teacher_kind;

  // the id of pair i of row t, -1 outside the vocabulary
  __device__ __forceinline__ int id(int64_t t, int i) const {
    const int64_t at = t * ld_ids + i;
    const int64_t v = id_bits == 64 ? __ldg(static_cast<const long long*>(ids) + at) : int64_t(__ldg(static_cast<const int*>(ids) + at));
    return v >= 0 && v < rows ? int(v) : -1;
  }
  __device__ __forceinline__ float logit(int64_t t, int i) const {
    const int64_t at = t * ld_teacher + i;
    return teacher_kind == BQ_ROWS_FP32 ? __ldg(static_cast<const float*>(teacher) + at)
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(teacher)[at]);
  }
  // a pair counts if its id is a word and the teacher gives it any weight; l: its logit
  __device__ __forceinline__ int kept_id(int64_t t, int i, float* l) const {
    const int v = id(t, i);
    *l = 0.f;
    if (!teacher || v < 0) return v;
    *l = logit(t, i);
    return *l == -INFINITY ? -1 : v;
  }
  // scale * (l - top).  The difference first, of halves: products of finite logits and the factor may overflow (a
  // row of the type's lowest value), and so may differences of them.
  __device__ __forceinline__ float behind(float l, float top) const { return 2.f * (scale * (0.5f * l - 0.5f * top)); }
};

// the teacher's softmax over a row's pairs, by a warp: the logit whose product with the factor is largest and the
// log of its sum; false if no pair counts
__device__ __forceinline__ bool teacher_sum(const Targets& y, int64_t t, int lane, float* top, float* log_sum) {
  const float sign = y.scale < 0.f ? -1.f : 1.f;
  float m = -INFINITY, l;
  bool any = false;
  for (int i = lane; i < y.k; i += 32)
    if (y.kept_id(t, i, &l) >= 0) any = true, m = fmaxf(m, sign * l);
  m = sign * warp_max(m);
  float s = 0.f;
  for (int i = lane; i < y.k; i += 32)
    if (y.kept_id(t, i, &l) >= 0) s += expf(y.behind(l, m));
  *top = m;
  *log_sum = logf(warp_sum(s));
  return __any_sync(0xFFFFFFFFu, any);
}

// ---------------------------------------------------------------- forward

struct PickArgs {
  const uint8_t *x, *w;
  const float *xs, *ws;
  float* out;
  int64_t ldx, ld_xs, ldw, ld_out, n;
  int cols;
  Targets y;
};

// The logits of words v[0 .. P) in row t, by a warp, the same in every lane: a lane takes 16 codes of each
// 512.  X's are decoded once for all P, and two steps' loads set out together.  (Bound by instructions, the
// decoding above all, where P is 1: 262144 pairs of 4096 codes took 275 us with a word a warp.)
template <int P>
__device__ __forceinline__ void picked(const PickArgs& g, int64_t t, const int (&v)[P], int lane, float (&z)[P]) {
  constexpr int STEPS = P == 1 ? 4 : 2;
  const uint8_t* x = g.x + t * g.ldx;
  const float* xs = g.xs + t;
  const int tile_cols = (g.cols + 127) / 128;
  float sum[P] = {};
  for (int c0 = 16 * lane; c0 < g.cols; c0 += 512 * STEPS) {
    uint4 a[STEPS], b[STEPS][P];
#pragma unroll
    for (int e = 0; e < STEPS; ++e) {
      const int c = c0 + 512 * e;
      if (c >= g.cols) continue;
      a[e] = __ldg(reinterpret_cast<const uint4*>(x + c));
#pragma unroll
      for (int i = 0; i < P; ++i) b[e][i] = __ldg(reinterpret_cast<const uint4*>(g.w + int64_t(v[i]) * g.ldw + c));
    }
#pragma unroll
    for (int e = 0; e < STEPS; ++e) {
      const int c = c0 + 512 * e;
      if (c >= g.cols) continue;
      const float f = __ldg(xs + int64_t(c >> 7) * g.ld_xs);
      float u[16];
      decode16(a[e], u);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float w[16];
        decode16(b[e][i], w);
        float2 d = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 16; j += 2) d = fma2(make_float2(u[j], u[j + 1]), make_float2(w[j], w[j + 1]), d);
        sum[i] = fmaf(d.x + d.y, f * __ldg(g.ws + int64_t(v[i] >> 7) * tile_cols + (c >> 7)), sum[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) z[i] = g.y.scale * warp_sum(sum[i]);
}

// Where the teacher's words are many, their logits are taken from the tiles of the product (kTilePicks) that holds
// them anyway; this sorts each row's words and finds where each part of the vocabulary begins.  4096 tokens
// of 32000 x 4096, 64 words each: 499 us in all so, 605 by k_loss_pick; 16 words each: 478 and 465.
struct SortArgs {
  Targets y;
  uint32_t* records;  // [parts + 1][ld]
  uint16_t* words;    // [n][k]
  int64_t n, ld;
  int parts;
};
constexpr int kSortFew = 256;  // words of a row at most, of 16 rows a CTA; of 4 rows kMaxPairs
constexpr int kSortSlots = 16 * (kSortFew + 1);
static_assert(4 * (kMaxPairs + 1) <= kSortSlots && 10 * kSortSlots <= 48 * 1024, "a CTA's words");

__global__ void __launch_bounds__(1024) k_loss_sort(const SortArgs g) {
  __shared__ int ids[kSortSlots], sorted[kSortSlots];
  __shared__ uint16_t order[kSortSlots];
  after_previous();
  next_may_start();
  const int k = g.y.k, pitch = k + 1, group = k <= kSortFew ? 16 : 4;
  const int64_t t0 = int64_t(blockIdx.x) * group;
  for (int i = threadIdx.x; i < group * k; i += 1024) {
    const int r = i / k, j = i - r * k;
    const int v = t0 + r < g.n ? g.y.id(t0 + r, j) : -1;
    ids[r * pitch + j] = v < 0 ? INT_MAX : v;  // (last, in no part)
  }
  __syncthreads();
  for (int i = threadIdx.x; i < group * k; i += 1024) {
    const int r = i / k, j = i - r * k, v = ids[r * pitch + j];
    int rank = 0;
    for (int e = 0; e < k; ++e) {
      const int x = ids[r * pitch + e];
      rank += x < v || (x == v && e < j);
    }
    sorted[r * pitch + rank] = v, order[r * pitch + rank] = uint16_t(j);
    if (t0 + r < g.n) g.words[(t0 + r) * k + rank] = uint16_t(j << 6 | (v & 63));
  }
  __syncthreads();
  // lanes along the rows: the place of row r's first word from 64 w on
  const int r = int(threadIdx.x) % group;
  if (t0 + r >= g.n) return;
  const int* mine = sorted + r * pitch;
  auto place = [&](int w) {
    int lo = 0, hi = k;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (mine[mid] < w * kPartCols)
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo;
  };
  // (a thread's parts one after another, so that each search is one)
  const int threads = 1024 / group, each = (g.parts + 1 + threads - 1) / threads;
  const int w0 = int(threadIdx.x) / group * each, w1 = min(w0 + each, g.parts + 1);
  int at = w0 < w1 ? place(w0) : 0;
  for (int w = w0; w < w1; ++w) {
    int next = at;
    while (next < k && mine[next] < (w + 1) * kPartCols) ++next;
    const uint32_t first = next > at ? uint32_t(order[r * pitch + at]) << 6 | uint32_t(mine[at] & 63) : 0u;
    g.records[int64_t(w) * g.ld + t0 + r] = words_record(uint32_t(at), uint32_t(next - at), first);
    at = next;
  }
}

// The logits of the teacher's words, four a warp, by reading their rows of W: bound by those bytes.
__global__ void __launch_bounds__(256) k_loss_pick(const PickArgs g) {
  after_previous();
  next_may_start();
  constexpr int P = 4;
  const int lane = threadIdx.x & 31, per_row = (g.y.k + P - 1) / P;
  const int64_t items = g.n * per_row, step = int64_t(gridDim.x) * 8;
  for (int64_t p = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); p < items; p += step) {
    const int64_t t = p / per_row;
    const int i0 = P * int(p - t * per_row);
    int v[P];
    bool any = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int id = i0 + i < g.y.k ? g.y.id(t, i0 + i) : -1;  // (what a pair without a word gets is not read)
      any |= id >= 0;
      v[i] = max(id, 0);
    }
    float z[P] = {};
    if (any) picked<P>(g, t, v, lane, z);
    if (lane < P && i0 + lane < g.y.k) g.out[t * g.ld_out + i0 + lane] = lane == 0 ? z[0] : lane == 1 ? z[1] : lane == 2 ? z[2] : z[3];
  }
}

struct JoinArgs {
  const float2* stats;
  const uint8_t* at;
  int64_t ld_stats, n, ld_logp;
  float *loss, *lse, *logp;  // logp holds the targets' logits; a class's is taken here
  int parts, group;  // group: rows of a CTA, 1, 2, .. kJoinWarps
  PickArgs pick;
};

__device__ __forceinline__ RowStats shuffled(const RowStats& a, int d) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.m, d), __shfl_xor_sync(0xFFFFFFFFu, a.s, d), __shfl_xor_sync(0xFFFFFFFFu, a.at, d)};
}

// A row's statistics from its parts', its log-sum, and its loss.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(32 * kJoinWarps) k_loss_join(const JoinArgs g) {
  __shared__ float sm[kJoinWarps][kJoinWarps + 1], ss[kJoinWarps][kJoinWarps + 1];
  __shared__ int sa[kJoinWarps][kJoinWarps + 1];
  after_previous();
  next_may_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Targets& y = g.pick.y;
  const int r = lane & (g.group - 1), each = 32 / g.group;
  const int64_t row = int64_t(blockIdx.x) * g.group + r, t = int64_t(blockIdx.x) * g.group + warp;
  const bool mine = warp < g.group && t < g.n;  // the row that this warp finishes
  float z = 0.f;
  int v = -1;
  if (!y.teacher && mine) {
    v = y.id(t, 0);
    if (v >= 0) {
      const int one[1] = {v};
      float got[1];
      picked<1>(g.pick, t, one, lane, got);
      z = got[0];
    }
  }
  RowStats a{-INFINITY, 0.f, 0};
  bool some = false;
  if (row < g.n)
    for (int p0 = warp * each + lane / g.group; p0 < g.parts; p0 += 4 * kJoinWarps * each) {
      float2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = p0 + e * kJoinWarps * each;
        if (p < g.parts) v[e] = g.stats[int64_t(p) * g.ld_stats + row];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = p0 + e * kJoinWarps * each;
        if (p >= g.parts) continue;
        const RowStats b{v[e].x, v[e].y, p};
        a = some ? joined(a, b) : b;
        some = true;
      }
    }
  // (a lane without a part holds the statistics of one logit of -inf, which add exp(-inf))
  for (int d = g.group; d < 32; d <<= 1) a = joined(a, shuffled(a, d));
  if (lane < g.group) sm[warp][lane] = a.m, ss[warp][lane] = a.s, sa[warp][lane] = a.at;
  __syncthreads();
  if (!mine) return;
  a = {sm[lane % kJoinWarps][warp], ss[lane % kJoinWarps][warp], sa[lane % kJoinWarps][warp]};
#pragma unroll
  for (int d = 1; d < kJoinWarps; d <<= 1) a = joined(a, shuffled(a, d));
  // (an infinite logit that is the maximum is inf - inf behind it, as any other: no word is the best)
  const int best = isinf(a.m) ? -1 : a.at * kPartCols + int(g.at[int64_t(a.at) * g.ld_stats + t]);
  const float more = log1pf(a.s);
  if (lane == 0) g.lse[t] = a.m + more;
  if (!y.teacher) {
    if (lane == 0) g.loss[t] = v < 0 ? 0.f : v == best ? more : more + (a.m - z);
    return;
  }
  float top, log_sum, sum = 0.f;
  const bool any = teacher_sum(y, t, lane, &top, &log_sum);
  for (int i = lane; i < y.k; i += 32) {
    v = y.kept_id(t, i, &z);
    float* at = g.logp + t * g.ld_logp + i;
    const float logp = v < 0 ? 0.f : v == best ? -more : (*at - a.m) - more;
    *at = logp;
    if (v < 0) continue;
    const float log_q = y.behind(z, top) - log_sum, q = expf(log_q);
    if (q != 0.f) sum += q * (log_q - logp);
  }
  sum = warp_sum(sum);
  if (lane == 0) g.loss[t] = any ? sum : 0.f;
}

// ---------------------------------------------------------------- gradient: operands

constexpr int kPrepCtas = 304;
constexpr int kHeadroom = 5;  // values of 448 x the largest scale below 2^15

// 2^e that brings 448 x `top` into [2^13, 2^15): fp16 holds what it scales
__device__ __forceinline__ int power_for(float top) {
  return top > 0.f ? max(-126, min(126, kHeadroom - ilogbf(top))) : 0;
}

struct PrepArgs {
  Targets y;
  const float *xs, *ws, *lse, *dloss;
  float *off, *tops;  // off: a row's log-sum, or kNoTarget; tops: each CTA's largest scale of X and of W
  int* target;        // a class, -1 for none
  int64_t ld_xs, n, w_tiles;
  int groups;
};

__device__ __forceinline__ float finite_abs(float v) {
  v = fabsf(v);
  return v <= 3.402823e38f ? v : 0.f;
}

// which rows have a target, and the largest scales
__global__ void __launch_bounds__(256) k_loss_prep(const PrepArgs g) {
  __shared__ float top[2][8];
  after_previous();
  next_may_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float mx = 0.f, mw = 0.f;
  for (int64_t t = int64_t(blockIdx.x) * 8 + warp; t < g.n; t += int64_t(gridDim.x) * 8) {
    // (loads that need nothing of one another set out together)
    const float f = g.dloss[t], lse = g.lse[t];
    float x = lane < g.groups ? finite_abs(g.xs[int64_t(lane) * g.ld_xs + t] * f) : 0.f;
    bool any = false;
    for (int i = lane; i < g.y.k; i += 32) {
      float z;
      any |= g.y.kept_id(t, i, &z) >= 0;
    }
    any = __any_sync(0xFFFFFFFFu, any);
    if (lane == 0) {
      // (an infinite log-sum: an infinite logit, or all -inf, and no softmax)
      g.off[t] = !any ? kNoTarget : isinf(lse) ? nanf("") : lse;
      g.target[t] = g.y.teacher ? -1 : g.y.id(t, 0);
    }
    if (!any) continue;
    for (int j = lane + 32; j < g.groups; j += 32) x = fmaxf(x, finite_abs(g.xs[int64_t(j) * g.ld_xs + t] * f));
    mx = fmaxf(mx, x);
  }
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < g.w_tiles; i += int64_t(gridDim.x) * 256)
    mw = fmaxf(mw, finite_abs(g.ws[i]));
  mx = warp_max(mx), mw = warp_max(mw);
  if (lane == 0) top[0][warp] = mx, top[1][warp] = mw;
  __syncthreads();
  if (threadIdx.x < 2) {
    float m = 0.f;
    for (int i = 0; i < 8; ++i) m = fmaxf(m, top[threadIdx.x][i]);
    g.tops[threadIdx.x * kPrepCtas + blockIdx.x] = m;
  }
}

// every thread of a CTA of 256: the largest of `count` values
__device__ __forceinline__ float largest(const float* v, int count) {
  __shared__ float top[8];
  float m = 0.f;
  for (int i = threadIdx.x; i < count; i += 256) m = fmaxf(m, v[i]);
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  m = top[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, top[i]);
  return m;
}

// fp16 rows of X, each times its loss's gradient (rows without a target: zeros, whatever they hold),
// or of W (off NULL)
struct HalfArgs {
  const uint8_t* codes;
  const float *scale, *off, *dloss, *tops;
  __half* out;
  float* back;  // the factor that takes the power of two back
  int64_t ldc, lds, ldo, n;
  int cols, count, ctas;
};

// A warp takes up to 1024 codes of a row, a lane 8 of each 256, so that loads and stores are whole lines;
// bound by memory (32256 x 4096: 58 us, 396 MB; 75 with 16 codes a lane).
__device__ __forceinline__ void half_rows(const HalfArgs& g, int cta) {
  const int lane = threadIdx.x & 31, spans = (g.cols + 1023) / 1024;
  const int64_t items = g.n * spans, step = int64_t(g.ctas) * 8;
  int64_t i = int64_t(cta) * 8 + (threadIdx.x >> 5), t = 0;
  int c0 = 0;
  uint2 q[4];
  float f[4], row = 1.f;
  bool none = false;
  auto load = [&] {
    t = i / spans;
    c0 = 1024 * int(i - t * spans) + 8 * lane;
    none = g.off && __ldg(g.off + t) == kNoTarget;
    row = g.off ? __ldg(g.dloss + t) : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 256 * k;
      if (c >= g.cols) continue;
      q[k] = __ldg(reinterpret_cast<const uint2*>(g.codes + t * g.ldc + c));
      f[k] = __ldg(g.off ? g.scale + int64_t(c >> 7) * g.lds + t : g.scale + (t >> 7) * g.lds + (c >> 7));
    }
  };
  if (i < items) load();  // (beside the search for the largest)
  const int e = power_for(largest(g.tops, g.count));
  const float up = ldexpf(1.f, e);
  if (cta == 0 && threadIdx.x == 0) *g.back = ldexpf(1.f, -e);
  while (i < items) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 256 * k;
      if (c >= g.cols) continue;
      const uint32_t w[2] = {q[k].x, q[k].y};
      uint32_t o[4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3)));
        const float s = (f[k] * row) * up;  // (in this order: the power of two is the products')
        if (!none) o[j] = two16(v.x * s, v.y * s, __half());
      }
      *reinterpret_cast<uint4*>(g.out + t * g.ldo + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if ((i += step) < items) load();
  }
}

// X's (x.ctas CTAs of the launch, 0: none) and a piece of W's
__global__ void __launch_bounds__(256) k_loss_half(const HalfArgs x, const HalfArgs w) {
  after_previous();
  next_may_start();
  if (int(blockIdx.x) < x.ctas)
    half_rows(x, int(blockIdx.x));
  else
    half_rows(w, int(blockIdx.x) - x.ctas);
}

struct FixArgs {
  Targets y;
  const float *off, *logp;
  __half* u;
  int64_t ldu, ld_logp, n;
  int v0, len;
};

// U at a teacher's words in a piece of the vocabulary: p - q by the forward pass's log-probability.  Where p is
// above 1/2 it is the others' weights less 1 - p, which keeps what is left of it where p and q are near 1, below
// it p - q itself, which keeps it where they are small (a class's is put into its tile, loss_tile.h)
__global__ void __launch_bounds__(128) k_loss_fix(const FixArgs g) {
  __shared__ float sq[4][kMaxPairs];
  __shared__ int sid[4][kMaxPairs];
  after_previous();
  next_may_start();
  const float unit = float(1 << kProbBits);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * 4 + warp;
  if (t >= g.n || g.off[t] == kNoTarget) return;
  float top, log_sum;
  teacher_sum(g.y, t, lane, &top, &log_sum);
  for (int i = lane; i < g.y.k; i += 32) {
    float z;
    const int v = g.y.kept_id(t, i, &z);
    sid[warp][i] = v;
    sq[warp][i] = v < 0 ? 0.f : expf(g.y.behind(z, top) - log_sum);
  }
  __syncwarp();
  for (int i = lane; i < g.y.k; i += 32) {
    const int id = sid[warp][i], v = id - g.v0;
    if (id < 0 || v < 0 || v >= g.len) continue;
    float q = 0.f, others = 0.f;  // (the same sums, in the same order, for every pair of this id)
    for (int j = 0; j < g.y.k; ++j) {
      const float w = sq[warp][j];
      if (sid[warp][j] == id)
        q += w;
      else
        others += w;
    }
    const float logp = g.logp[t * g.ld_logp + i];
    others += 0.f * q;  // (a weight that is NaN)
    g.u[t * g.ldu + v] = __float2half_rn(unit * (logp > -0.6931472f ? expm1f(logp) + others : expf(logp) - q));
  }
}

// ---------------------------------------------------------------- gradient: few tokens
// dX of few tokens: U as the sum of three E4M3 values, whose products with W's codes are an FP8
// projection (k_linear, transposed) of three rows a token, 42 tokens a tile of 128.  It reads W as it is,
// where fp16 operands are written and read: 16 tokens of 128256 x 4096 take 103 us so (W's bytes alone 78),
// and 505 by fp16 pieces.
constexpr int kTokensOfTile = 42;
int64_t triple_rows(int64_t n) { return n / kTokensOfTile * 128 + 3 * (n % kTokensOfTile); }

struct SplitArgs {
  const __half* u;
  uint8_t* codes;  // rows as triple_rows counts them
  float* scale;    // [groups][lds]
  int64_t ldu, ldc, lds;
  int n, len;
};

// A warp takes 128 values of a token.  The scales are powers of two, 2^4 apart: what a term leaves
// (16 of its scales at most, half the largest step) is 256 of the next one's, and what the third leaves is below
// 2^-12 of the value, or 2^-25 of the group's largest (half the smallest step, 2^-10, of a scale that is
// 2^-8 of the first, the largest being 224 of the first or more).
__global__ void __launch_bounds__(256) k_loss_split(const SplitArgs g) {
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31, groups = (g.len + 127) / 128;
  const int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= int64_t(g.n) * groups) return;
  const int t = int(i / groups), j = int(i - int64_t(t) * groups), c = 128 * j + 4 * lane;
  // (whole words: U's pitch covers them)
  const uint2 q = c < g.ldu ? *reinterpret_cast<const uint2*>(g.u + t * g.ldu + c) : make_uint2(0u, 0u);
  float2 v[2] = {__half22float2(*reinterpret_cast<const __half2*>(&q.x)), __half22float2(*reinterpret_cast<const __half2*>(&q.y))};
  if (c >= g.len) v[0].x = 0.f;
  if (c + 1 >= g.len) v[0].y = 0.f;
  if (c + 2 >= g.len) v[1].x = 0.f;
  if (c + 3 >= g.len) v[1].y = 0.f;
  float top = warp_max(fmaxf(fmaxf(fabsf(v[0].x), fabsf(v[0].y)), fmaxf(fabsf(v[1].x), fabsf(v[1].y))));
  // 2^e, e the least with top <= 448 * 2^e (top is an fp16 value: 2^-24 at least unless it is 0)
  int e0 = top > 0.f && top <= 65504.f ? ilogbf(top) - 8 : 0;
  if (top > ldexpf(448.f, e0)) ++e0;
  const int64_t row = int64_t(t / kTokensOfTile) * 128 + 3 * (t % kTokensOfTile);
  float s = ldexpf(1.f, e0), back = ldexpf(1.f, -e0);
#pragma unroll
  for (int term = 0; term < 3; ++term) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const __nv_fp8x2_storage_t code = __nv_cvt_float2_to_fp8x2(mul2(v[e], dup(back)), __NV_SATFINITE, __NV_E4M3);
      const float2 d = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3)));
      v[e] = fma2(d, dup(-s), v[e]);  // (exact)
      w |= uint32_t(code) << (16 * e);
    }
    if (c < g.ldc) *reinterpret_cast<uint32_t*>(g.codes + (row + term) * g.ldc + c) = w;
    if (lane == 0) g.scale[int64_t(j) * g.lds + row + term] = top <= 65504.f ? s : top;
    s *= 0.0625f, back *= 16.f;
  }
}

// ---------------------------------------------------------------- gradient: dX = U W
// On CTA pairs, 256 x 256 tiles, fp16 operands and fp32 sums: U's rows K-major, W's words
// MN-major.  Tiles left over after whole waves of pairs are cut into `parts` equal parts of their
// summed index, taken in turn by all pairs, a part of every tile before the next part: 28 tiles left
// of 256 on 76 pairs take three rounds of an eighth, not a wave (4096 x 32256 x 4096: 575 us, 633 with
// whole tiles).  Cutting them into as many pieces as there are pairs, each pair's at an offset of its own, balances them
// exactly and took 6 % longer than equal parts: pairs at different offsets read nothing that others have read.
// Sums of a tile leave as shares, one per part, which pieces of the vocabulary add to; k_loss_sums
// adds a tile's shares in order.
//
// W's fp16 words come from a launch before (k_loss_half).  Spreading its codes to fp16 inside
// this kernel, by six warps between a ring of codes and the products' operands, took 1225 us where
// this and that launch take 633 (4096 x 32256 x 4096): 250 of it the spreading, 130 its fences and cluster-wide
// arrivals, and 815 were left without both.

// Which tiles, and which parts of their k-blocks, a pair works on: its share of the whole waves'
// tiles, then of the parts of those left.
struct Shares {
  int tiles, whole, parts;

  __host__ __device__ int left() const { return tiles - whole; }
  // where a tile's share of a part is kept, in tiles
  __host__ __device__ int at(int tile, int part) const { return part == 0 ? tile : tiles + (part - 1) * left() + tile - whole; }
  __host__ __device__ int64_t kept() const { return tiles + int64_t(parts - 1) * left(); }
};

struct DxArgs {
  float* part;
  const float *row_factor, *off, *back;  // back: takes back W's power of two
  __nv_bfloat16* out;
  float factor;
  int64_t ldo;
  int m, n, k;          // tokens, columns, words
  int add;
  Shares sh;
  int* status;
};

// piece of work i of a pair: false after the last
__device__ __forceinline__ bool dx_segment(const Shares& sh, int pair, int npairs, int nk, int i, int& tile, int& at, int& k0, int& k1) {
  const int t = pair + i * npairs;
  if (t < sh.whole) {
    tile = at = t, k0 = 0, k1 = nk;
    return true;
  }
  const int r = t - sh.whole, part = sh.left() ? r / sh.left() : sh.parts;
  if (part >= sh.parts) return false;
  tile = sh.whole + r - part * sh.left();
  at = sh.at(tile, part);
  k0 = int(int64_t(nk) * part / sh.parts), k1 = int(int64_t(nk) * (part + 1) / sh.parts);
  return true;
}

// Instruction descriptor, kind::f16: D fp32 (bits 4-5 = 1), A and B fp16 (0), majors in bits 15, 16
__host__ __device__ constexpr uint32_t product_idesc(bool a_k_major) {
  return (1u << 4) | (uint32_t(!a_k_major) << 15) | (1u << 16) | (uint32_t(PN >> 3) << 17) | (uint32_t(PM >> 4) << 24);
}

__global__ void __launch_bounds__(PAIR_THREADS, 1)
    k_loss_dx(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const DxArgs g) {
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
  const int mt = (g.m + PM - 1) / PM, nt = (g.n + PN - 1) / PN;
  const int nk = (g.k + DK - 1) / DK;
  const int pair = int(blockIdx.x >> 1), npairs = int(gridDim.x >> 1);
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

  int tile, at, k0, k1;
  if (warp == 0) {
    // ---------------- TMA producer (both CTAs: this CTA's halves)
    uint32_t it = 0;
    bool ok = true;
    for (int i = 0; ok && dx_segment(g.sh, pair, npairs, nk, i, tile, at, k0, k1); ++i) {
      int bm, bn;
      banded_tile(tile, mt, nt, kBand, bm, bn);
      const int ma = bm * PM + 128 * rank, nb = bn * PN + 128 * rank;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(empty_bar(s), ((it / DW_STAGES) & 1u) ^ 1u, g.status, 61);
        if (!ok) break;
        const uint32_t a_dst = base + uint32_t(s) * PSTAGE_BYTES, b_dst = a_dst + HALF_STAGE;
        const uint32_t fb = map_rank(full_bar(s), 0);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full_bar(s), 2 * PSTAGE_BYTES);
          tma_load_2d_pair(a_dst, &tmA, kb * DK * 2, ma, fb);  // (the map counts bytes)
          tma_load_3d_pair(b_dst, &tmB, kb * DK, nb / 64, fb);
        }
        __syncwarp();
      }
    }
    // drain (leader): the pair's last copies have landed; the peer waits for this at
    // the closing cluster barrier
    if (rank == 0)
      for (uint32_t d = it > uint32_t(DW_STAGES) ? it - DW_STAGES : 0; d < it; ++d)
        mbar_wait(full_bar(int(d % DW_STAGES)), (d / DW_STAGES) & 1u, g.status, 62);
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer (leader)
    uint32_t it = 0, tc = 0;
    bool ok = true;
    for (int i = 0; ok && dx_segment(g.sh, pair, npairs, nk, i, tile, at, k0, k1); ++i) {
      if (k0 == k1) continue;
      const int buf = int(tc & 1u);
      if (tc >= 2) ok = mbar_wait_cluster_relaxed(tempty_bar(buf), ((tc >> 1) & 1u) ^ 1u, g.status, 63);
      if (!ok) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(full_bar(s), (it / DW_STAGES) & 1u, g.status, 64);
        if (!ok) break;
        tc_fence_after();
        // 16 words a product: U's rows 32 bytes on, W's 2 KB (64-column chunks 8 KB apart)
        const uint32_t a_addr = base + uint32_t(s) * PSTAGE_BYTES;
        const uint64_t ad = sdesc(a_addr, 16, 1024), bd = sdesc(a_addr + HALF_STAGE, CHUNK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_pair(tmem + uint32_t(buf) * PN, ad + uint64_t(2 * kk), bd + uint64_t(128 * kk),
                          product_idesc(true), kb != k0 || kk != 0 ? 1u : 0u);
          mma_commit_pair(empty_bar(s));
          if (kb + 1 == k1) mma_commit_pair(tfull_bar(buf));
        }
        __syncwarp();
      }
      if (ok) ++tc;
    }
    // every product issued here has finished before the accumulators are freed
    if (tc > 0 && ok) mbar_wait(tfull_bar(int((tc - 1) & 1u)), ((tc - 1) >> 1) & 1u, g.status, 66);
  } else if (warp >= 4) {
    // ---------------- shares (both CTAs: this CTA's 128 rows)
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t te0 = map_rank(tempty_bar(0), 0);
    uint32_t tc = 0;
    for (int i = 0; dx_segment(g.sh, pair, npairs, nk, i, tile, at, k0, k1); ++i) {
      if (k0 == k1 && g.add) continue;
      int bm, bn;
      banded_tile(tile, mt, nt, kBand, bm, bn);
      const int row0 = bm * PM + 128 * rank + 32 * q, c0 = bn * PN + PCOLS * part;
      uint32_t r[PCOLS];
      if (k0 < k1) {
        const uint32_t buf = tc & 1u;
        if (!mbar_wait(tfull_bar(int(buf)), (tc >> 1) & 1u, g.status, 65)) break;
        tc_fence_after();
        const uint32_t from = tmem + (uint32_t(32 * q) << 16) + buf * PN + uint32_t(PCOLS * part);
        tmem_ld32(from, r);
        tmem_ld32(from + 32, r + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(te0 + 8u * buf);
        ++tc;
      } else {  // (no k-block of this piece: the share begins as zeros)
#pragma unroll
        for (int j = 0; j < PCOLS; ++j) r[j] = 0u;
      }
      if (row0 >= g.m || c0 >= g.n) continue;
      float4* o = reinterpret_cast<float4*>(g.part) + share_at(at, rank, warp - 4) + lane;
#pragma unroll
      for (int j = 0; j < PCOLS / 4; ++j) {
        float4 v = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                               __uint_as_float(r[4 * j + 3]));
        if (g.add) {
          const float4 x = o[32 * j];
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        o[32 * j] = v;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmem);
  }
}
static_assert(2 * DW_SMEM > kSmemOfSm && DW_SMEM >= kClusterSmemLeast, "a pair's CTA has its SM's tensor memory to itself");

// 16 values of a row of a sum of shares, rounded to out (+ out)
__device__ __forceinline__ void put16(const float* x, __nv_bfloat16* o, bool aligned, bool accumulate) {
  alignas(16) __nv_bfloat16 y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = __float2bfloat16_rn(accumulate ? x[e] + __bfloat162float(o[e]) : x[e]);
  if (aligned) {
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(y);
    *reinterpret_cast<uint4*>(o + 8) = *reinterpret_cast<const uint4*>(y + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = y[e];
  }
}

// ---------------------------------------------------------------- gradient: dW = U^T X
// The weight gradient of a projection (k_dw_pair) with fp16 operands, out times a factor: bound by
// the tensor cores, for few tokens by the stores.

struct DwPieceArgs {
  __nv_bfloat16* out;
  float* part;        // shares of the sum [splits][tiles], or NULL
  const float* back;  // takes back X's power of two
  float factor;
  int64_t ldo;
  int m, n, k;        // words, columns, tokens
  int splits, accumulate, bytes;
  int late;           // the launch before is dx's, which this one does not need: it waits for its end at its own
  int* status;
};

__global__ void __launch_bounds__(PAIR_THREADS, 1)
    k_loss_dw(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO, const DwPieceArgs g) {
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
  const int mt = (g.m + PM - 1) / PM, nt = (g.n + PN - 1) / PN, ntiles = mt * nt, total = ntiles * g.splits;
  const int nk = (g.k + DK - 1) / DK;
  const int pair = int(blockIdx.x >> 1), npairs = int(gridDim.x >> 1);
  // tile t: share t / ntiles of the k-blocks [k0, k1)
  auto tile_of = [&](int t, int& bm, int& bn, int& k0, int& k1) {
    const int sp = t / ntiles;
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
  if (!g.late) after_previous();
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
      int bm, bn, k0, k1;
      tile_of(t, bm, bn, k0, k1);
      const int ma = bm * PM + 128 * rank, nb = bn * PN + 128 * rank;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(empty_bar(s), ((it / DW_STAGES) & 1u) ^ 1u, g.status, 51);
        if (!ok) break;
        const uint32_t a_dst = base + uint32_t(s) * PSTAGE_BYTES, b_dst = a_dst + HALF_STAGE;
        const uint32_t fb = map_rank(full_bar(s), 0);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full_bar(s), 2 * PSTAGE_BYTES);
          tma_load_3d_pair(a_dst, &tmA, kb * DK, ma / 64, fb);
          tma_load_3d_pair(b_dst, &tmB, kb * DK, nb / 64, fb);
        }
        __syncwarp();
      }
    }
    // drain (leader): the pair's last copies have landed; the peer waits for this at
    // the closing cluster barrier
    if (rank == 0)
      for (uint32_t d = it > uint32_t(DW_STAGES) ? it - DW_STAGES : 0; d < it; ++d)
        mbar_wait(full_bar(int(d % DW_STAGES)), (d / DW_STAGES) & 1u, g.status, 52);
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer (leader)
    uint32_t it = 0, tc = 0;
    bool ok = true;
    for (int t = pair; ok && t < total; t += npairs) {
      int bm, bn, k0, k1;
      tile_of(t, bm, bn, k0, k1);
      const int buf = int(tc & 1u);
      if (tc >= 2) ok = mbar_wait_cluster_relaxed(tempty_bar(buf), ((tc >> 1) & 1u) ^ 1u, g.status, 53);
      if (!ok) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = int(it % DW_STAGES);
        ok = mbar_wait(full_bar(s), (it / DW_STAGES) & 1u, g.status, 54);
        if (!ok) break;
        tc_fence_after();
        // 64-column chunks 8 KB apart, 16 tokens (2 KB) a product
        const uint32_t a_addr = base + uint32_t(s) * PSTAGE_BYTES;
        const uint64_t ad = sdesc(a_addr, CHUNK, 1024), bd = sdesc(a_addr + HALF_STAGE, CHUNK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_pair(tmem + uint32_t(buf) * PN, ad + uint64_t(128 * kk), bd + uint64_t(128 * kk),
                          product_idesc(false), kb != k0 || kk != 0 ? 1u : 0u);
          mma_commit_pair(empty_bar(s));
          if (kb + 1 == k1) mma_commit_pair(tfull_bar(buf));
        }
        __syncwarp();
      }
      if (ok) ++tc;
    }
    // every product issued here has finished before the accumulators are freed
    if (tc > 0 && ok) mbar_wait(tfull_bar(int((tc - 1) & 1u)), ((tc - 1) >> 1) & 1u, g.status, 56);
  } else if (warp >= 4) {
    // ---------------- output (both CTAs: this CTA's 128 rows)
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t te0 = map_rank(tempty_bar(0), 0);
    const uint32_t box = base + DW_STAGES * PSTAGE_BYTES + uint32_t(warp - 4) * DW_BOX;
    const float back = g.part ? 1.f : __ldcg(g.back);
    uint32_t tc = 0;
    for (int t = pair; t < total; t += npairs, ++tc) {
      int bm, bn, k0, k1;
      tile_of(t, bm, bn, k0, k1);
      const uint32_t buf = tc & 1u;
      if (!mbar_wait(tfull_bar(int(buf)), (tc >> 1) & 1u, g.status, 55)) break;
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
        if (row0 < g.m && c0 < g.n)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[32 * j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                    __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
        continue;
      }
#pragma unroll
      for (int j = 0; j < 64; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * g.factor * back);
      if (g.accumulate && row < g.m) {
        // (from L2: this may have begun before the launch before ended)
        const auto* o = reinterpret_cast<const unsigned short*>(g.out + int64_t(row) * g.ldo + c0);
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (c0 + j < g.n) r[j] = __float_as_uint(__uint_as_float(r[j]) + bf16f(__ldcg(o + j)));
      }
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last box has been read
      __syncwarp();
      put_box<64>(reinterpret_cast<const float*>(r), box, lane);
      store_box<64>(g.out, g.ldo, g.m, g.n, g.bytes, &tmO, row0, c0, box, lane);
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
  if (g.late) after_previous();
}

// dx = the shares' sum in order, times its row's factor: warp i takes 32 rows x 16 columns
__device__ __forceinline__ void sum_dx(const DxArgs& g, int64_t i) {
  const int mt = (g.m + PM - 1) / PM, nt = (g.n + PN - 1) / PN;
  const int lane = threadIdx.x & 31, h = int(i & 3), w = int(i >> 2) & (PEPI - 1), rank = int(i >> 6) & 1, t = int(i >> 7);
  int bm, bn;
  banded_tile(t, mt, nt, kBand, bm, bn);
  const int row = bm * PM + 128 * rank + 32 * (w & 3) + lane, c0 = bn * PN + 64 * (w >> 2) + 16 * h;
  if (row >= g.m || c0 >= g.n) return;
  const int count = t < g.sh.whole ? 1 : g.sh.parts;
  float4 v[4] = {};
  for (int k = 0; k < count; ++k) {
    const float4* p = reinterpret_cast<const float4*>(g.part) + share_at(g.sh.at(t, k), rank, w) + 128 * h + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = p[32 * j];
      v[j].x += x.x, v[j].y += x.y, v[j].z += x.z, v[j].w += x.w;
    }
  }
  const bool none = __ldg(g.off + row) == kNoTarget;  // (whatever W holds)
  const float f = g.factor * __ldg(g.row_factor + row), f2 = __ldg(g.back);
  float* x = reinterpret_cast<float*>(v);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = none ? 0.f : x[e] * f * f2;
  put16(x, g.out + int64_t(row) * g.ldo + c0, g.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0, false);
}

// out = the shares' sum in order, times its factors (+ out): warp i takes 32 rows x 16 columns
__device__ __forceinline__ void sum_dw(const DwPieceArgs& g, int64_t i) {
  const int mt = (g.m + PM - 1) / PM, nt = (g.n + PN - 1) / PN, ntiles = mt * nt;
  const int lane = threadIdx.x & 31, h = int(i & 3), w = int(i >> 2) & (PEPI - 1), rank = int(i >> 6) & 1, t = int(i >> 7);
  int bm, bn;
  banded_tile(t, mt, nt, kBand, bm, bn);
  const int row = bm * PM + 128 * rank + 32 * (w & 3) + lane, c0 = bn * PN + 64 * (w >> 2) + 16 * h;
  if (row >= g.m || c0 >= g.n) return;
  const float4* p = reinterpret_cast<const float4*>(g.part) + share_at(t, rank, w) + 128 * h + lane;
  float4 v[4] = {};
  for (int k = 0; k < g.splits; ++k, p += share_at(ntiles, 0, 0))
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = p[32 * j];
      v[j].x += x.x, v[j].y += x.y, v[j].z += x.z, v[j].w += x.w;
    }
  const float back = __ldg(g.back);
  float* x = reinterpret_cast<float*>(v);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x[e] * g.factor * back;
  put16(x, g.out + int64_t(row) * g.ldo + c0, g.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0, g.accumulate);
}

// the first dx_ctas CTAs: dx's
__global__ void __launch_bounds__(256) k_loss_sums(const DxArgs dx, const DwPieceArgs dw, int dx_ctas) {
  after_previous();
  next_may_start();
  const int cta = int(blockIdx.x), warp = int(threadIdx.x >> 5);
  if (cta < dx_ctas)
    sum_dx(dx, int64_t(cta) * 8 + warp);
  else
    sum_dw(dw, int64_t(cta - dx_ctas) * 8 + warp);
}

// ---------------------------------------------------------------- host

constexpr size_t kStatus = 256;

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
size_t scale_bytes(int64_t n, int64_t cols) { return up(size_t((cols + 127) / 128) * size_t(up_to(n, 4)) * 4); }

struct ForwardWs {
  size_t scales, stats, at, records, words, bytes;
};

// k: a teacher's words taken from the tiles, 0 for none
ForwardWs forward_ws(int64_t n, int64_t rows, int64_t cols, int64_t k) {
  ForwardWs p;
  const size_t parts = size_t((rows + kPartCols - 1) / kPartCols);
  p.scales = kStatus;
  p.stats = p.scales + scale_bytes(n, cols);
  p.at = p.stats + up(parts * size_t(n) * 8);
  p.records = p.at + up(parts * size_t(n));
  p.words = p.records + (k ? up((parts + 1) * size_t(n) * 4) : 0);
  p.bytes = p.words + up(size_t(n) * size_t(k) * 2);
  return p;
}

// Whether a teacher's words are sorted and taken from the tiles, by the times of 32 losses: where three quarters of what
// reading their rows of W takes (5 TB/s) are more than the sort (10 us, 0.18 a word of a row, and its records) and 0.9 us
// a round of tiles for looking at the records.
bool from_tiles(int64_t n, int64_t rows, int64_t cols, int64_t k) {
  const double pick = double(n) * double(k) * double(cols) / 5e6, sort = 10 + 0.18 * double(k) + double(n) * double(rows) / 64 / 0.6e6;
  const double rounds = double((n + PM - 1) / PM) * double((rows + PN - 1) / PN) / cluster_slots()[2];
  return 0.75 * pick > sort + 0.9 * rounds && linear_whole_tiles(n, rows, cols);
}

struct GradWs {
  int64_t piece;      // words of a piece of the vocabulary, a multiple of 256
  int pieces;
  int64_t ldh;        // pitch of the fp16 rows of X
  bool few;           // dx by three E4M3 terms of U, whose codes and scales then lie at w and dx
  Shares dx_shares;
  size_t scales, tops, back, off, target, x, u, w, dx, dw, bytes;
};

int64_t piece_len(const GradWs& p, int64_t rows, int i) { return std::min(p.piece, rows - i * p.piece); }

// U takes 512 MB at most and the piece of W in fp16 1 GB, unless 256 words do not fit
constexpr int64_t kPieceBytes = int64_t(512) << 20, kPieceWeight = int64_t(1) << 30;

// The tiles left over after whole waves in the parts that cost least: a round of parts takes 0.29 us a k-block (as
// a projection's weight gradient), and a share is stored and added up.  us: what the product takes.
Shares dx_shares(int64_t n, int64_t cols, int64_t piece, double* us = nullptr) {
  Shares sh;
  const int pairs = cluster_slots()[2], nk = int((piece + DK - 1) / DK);
  sh.tiles = int(((n + PM - 1) / PM) * ((cols + PN - 1) / PN));
  sh.whole = sh.tiles / pairs * pairs;
  sh.parts = 1;
  const int left = sh.left();
  double least = 0;
  for (int parts = 1; left && parts <= std::min(nk, 64); ++parts) {
    const double t = 0.29 * ((nk + parts - 1) / parts) * ((left * parts + pairs - 1) / pairs) + parts * (0.25 + 0.045 * left);
    if (parts == 1 || t < least) least = t, sh.parts = parts;
  }
  if (us) *us = least + 0.29 * nk * (sh.whole / pairs);
  return sh;
}

// Whether dx takes three E4M3 terms of U: where splitting U (5 bytes a value at 4 TB/s) and the FP8 product of three
// rows a token cost less than W in fp16 (3 bytes a value at 6 TB/s) and its product.
bool few_tokens(int64_t n, int64_t rows, int64_t cols) {
  if (n * rows * 2 > kPieceBytes) return false;
  double us = 0;
  dx_shares(n, cols, rows, &us);
  return double(n) * double(rows) * 5 / 4e6 + linear_small_us(triple_rows(n), cols, rows) < double(rows) * double(cols) * 3 / 6e6 + 3 + us;
}

GradWs grad_ws(int64_t n, int64_t rows, int64_t cols) {
  GradWs p;
  p.ldh = up_to(cols, 64);
  p.few = few_tokens(n, rows, cols);
  const int64_t most = p.few ? up_to(rows, 256)
                              : std::max<int64_t>(256, std::min(kPieceBytes / std::max<int64_t>(n, 1), kPieceWeight / p.ldh) / 512 * 256);
  const int64_t pieces = (rows + most - 1) / most;
  p.piece = up_to((rows + pieces - 1) / pieces, 256);
  p.pieces = int((rows + p.piece - 1) / p.piece);
  p.dx_shares = dx_shares(n, cols, p.piece);
  p.scales = kStatus;
  p.tops = p.scales + scale_bytes(n, cols);
  p.back = p.tops + up(2 * kPrepCtas * 4);
  p.off = p.back + 256;
  p.target = p.off + up(size_t(n) * 4);
  p.x = p.target + up(size_t(n) * 4);
  p.u = p.x + up(size_t(n) * size_t(p.ldh) * 2);
  p.w = p.u + up(size_t(n) * size_t(p.piece) * 2);
  p.dx = p.w + up(p.few ? size_t(triple_rows(n)) * size_t(p.piece) : size_t(p.piece) * size_t(p.ldh) * 2);
  p.dw = p.dx + up(p.few ? size_t(p.piece / 128) * size_t(up_to(triple_rows(n), 4)) * 4 : size_t(p.dx_shares.kept()) * PM * PN * 4);
  size_t dw = 0;
  for (int i : {0, p.pieces - 1}) {
    const int64_t len = piece_len(p, rows, i);
    dw = std::max(dw, dw_part_bytes(dw_splits(n, len, cols), len, cols));
  }
  p.bytes = p.dw + dw;
  return p;
}

Targets targets(const LossArgs& a) {
  Targets y;
  y.ids = a.ids, y.teacher = a.teacher, y.ld_ids = a.ld_ids, y.ld_teacher = a.ld_teacher, y.scale = a.scale;
  y.rows = a.rows, y.k = a.k, y.id_bits = a.id_bits, y.teacher_kind = a.teacher_kind;
  return y;
}

unsigned ctas_for(int64_t items, int64_t each, int64_t most) {
  return unsigned(std::max<int64_t>(1, std::min<int64_t>(most, (items + each - 1) / each)));
}

}  // namespace

// (of a class or of any teacher)
size_t loss_bytes(int64_t n, int64_t rows, int64_t cols) { return forward_ws(n, rows, cols, kMaxPairs).bytes; }
size_t loss_grad_bytes(int64_t n, int64_t rows, int64_t cols) { return grad_ws(n, rows, cols).bytes; }

int launch_loss(const LossArgs& a, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto* base = static_cast<unsigned char*>(ws);
  const bool tiles = a.teacher && from_tiles(a.n, a.rows, a.cols, a.k);
  const ForwardWs p = forward_ws(a.n, a.rows, a.cols, tiles ? a.k : 0);
  PickArgs pick;
  pick.x = a.x, pick.w = a.w, pick.xs = a.x_scale, pick.ws = a.w_scale;
  pick.out = a.logp, pick.ld_out = a.ld_logp;
  pick.ldx = a.ldx, pick.ld_xs = a.ld_xs, pick.ldw = a.ldw, pick.n = a.n, pick.cols = a.cols;
  pick.y = targets(a);
  // the targets' logits beside the product, which reads nothing of theirs (but for a copy of X's scales, it is the
  // next launch)
  const bool pick_first = a.teacher && !tiles && (!linear_on_pairs(a.n, a.rows, a.cols) ||
                                        (a.ld_xs % 4 == 0 && (reinterpret_cast<uintptr_t>(a.x_scale) & 15) == 0));
  if (tiles) {
    SortArgs sort;
    sort.y = pick.y, sort.n = a.n, sort.parts = (a.rows + kPartCols - 1) / kPartCols;
    sort.records = reinterpret_cast<uint32_t*>(base + p.records), sort.ld = a.n, sort.words = reinterpret_cast<uint16_t*>(base + p.words);
    const int group = a.k <= kSortFew ? 16 : 4;
    launch_after(k_loss_sort, unsigned((a.n + group - 1) / group), 1024, 0, s, sort);
    if (int rc = check("loss (teacher's words)")) return rc;
  } else if (a.teacher) {
    launch_after(k_loss_pick, ctas_for(a.n * ((a.k + 3) / 4), 8, int64_t(sm_count()) * 64), 256, 0, s, pick);
    if (int rc = check("loss (targets)")) return rc;
  }
  LossTile tile = {};
  tile.end = tiles ? kTilePicks : kTileStats, tile.zscale = a.scale;
  tile.late = pick_first;
  tile.records = reinterpret_cast<uint32_t*>(base + p.records), tile.ld_records = a.n, tile.words = reinterpret_cast<uint16_t*>(base + p.words);
  tile.picked = a.logp, tile.ld_picked = a.ld_logp, tile.listed = a.k;
  tile.stats = reinterpret_cast<float2*>(base + p.stats), tile.at = base + p.at, tile.ld_stats = a.n;
  LinearArgs l{a.x, a.x_scale, a.w, a.w_scale, base, a.ldx, a.ld_xs, a.ldw, a.rows, a.n, a.rows, a.cols, 0,
               static_cast<int*>(ws), reinterpret_cast<float*>(base + p.scales), &tile};
  if (int rc = launch_linear_fp8(l, stream)) return rc;
  JoinArgs j;
  j.stats = tile.stats, j.at = tile.at, j.ld_stats = a.n, j.n = a.n, j.ld_logp = a.ld_logp;
  j.loss = a.loss, j.lse = a.lse, j.logp = a.logp;
  j.parts = (a.rows + kPartCols - 1) / kPartCols;
  j.group = 1;
  while (j.group < kJoinWarps && a.n > int64_t(j.group) * 2 * sm_count()) j.group *= 2;
  j.pick = pick;
  launch_after(k_loss_join, unsigned((a.n + j.group - 1) / j.group), 32 * kJoinWarps, 0, s, j);
  return check("loss (join)");
}

int launch_loss_grad(const LossArgs& a, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static OncePerDevice once;
  if (int rc = once.run(current_device(), [] {
        if (cudaFuncSetAttribute(k_loss_dx, cudaFuncAttributeMaxDynamicSharedMemorySize, DW_SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(k_loss_dw, cudaFuncAttributeMaxDynamicSharedMemorySize, DW_SMEM) != cudaSuccess)
          return check("loss gradient (shared memory attribute)");
        return int(BQ_OK);
      }))
    return rc;
  auto* base = static_cast<unsigned char*>(ws);
  const GradWs p = grad_ws(a.n, a.rows, a.cols);
  int* status = static_cast<int*>(ws);
  float *tops = reinterpret_cast<float*>(base + p.tops), *back = reinterpret_cast<float*>(base + p.back);
  float* off = reinterpret_cast<float*>(base + p.off);
  int* target = reinterpret_cast<int*>(base + p.target);
  auto *x16 = reinterpret_cast<__half*>(base + p.x), *u = reinterpret_cast<__half*>(base + p.u), *w16 = reinterpret_cast<__half*>(base + p.w);
  const int64_t tile_cols = (a.cols + 127) / 128;

  // X's scales as the pairs read them, copied once for all pieces
  const bool pairs = linear_on_pairs(a.n, piece_len(p, a.rows, 0), a.cols) || linear_on_pairs(a.n, piece_len(p, a.rows, p.pieces - 1), a.cols);
  const float* xs = a.x_scale;
  int64_t ld_xs = a.ld_xs;
  if (pairs && (ld_xs % 4 || (reinterpret_cast<uintptr_t>(xs) & 15))) {
    auto* to = reinterpret_cast<float*>(base + p.scales);
    if (int rc = launch_copy_scales(xs, ld_xs, a.n, tile_cols, to, up_to(a.n, 4), stream)) return rc;
    xs = to, ld_xs = up_to(a.n, 4);
  }
  PrepArgs prep;
  prep.y = targets(a);
  prep.xs = xs, prep.ws = a.w_scale, prep.lse = a.lse, prep.dloss = a.dloss, prep.off = off, prep.tops = tops, prep.target = target;
  prep.ld_xs = ld_xs, prep.n = a.n, prep.w_tiles = tile_cols * ((a.rows + 127) / 128), prep.groups = int(tile_cols);
  const int prep_ctas = int(ctas_for(std::max<int64_t>(a.n * 32, prep.w_tiles), 256, kPrepCtas));
  launch_after(k_loss_prep, unsigned(prep_ctas), 256, 0, s, prep);
  if (int rc = check("loss gradient (targets)")) return rc;

  const int64_t half_ctas = int64_t(sm_count()) * 16;
  CUtensorMap tx, tw, tu, to;
  HalfArgs hx = {}, hw = {};
  if (a.dw) {
    hx = {a.x, xs, off, a.dloss, tops, x16, back, a.ldx, ld_xs, p.ldh, a.n, a.cols, prep_ctas,
          int(ctas_for(a.n * ((a.cols + 1023) / 1024), 8, half_ctas))};
    if (int rc = encode_map_chunks(&tx, x16, a.cols, a.n, p.ldh, 2)) return rc;
  }
  const float unscale = a.scale * (1.f / float(1 << kProbBits));
  // dW beside dx.  Few tokens' dx is bound by memory, as dW is: of a large head they only slow each other (16 tokens of 128256 x
  // 4096: 363 us in turn, 372 beside; of 64000 x 4096: 196.6 and 198.5), of a small one dW hides its start (4 of 1298 x 608: 22.6
  // and 19.0; 16 of 8192 x 2048, 2^24 codes: 36.9 and 35.5).  Between 2^24 and 2^27 codes beside still gains 1 to 2 %
  // (16 of 32000 x 4096: 111.5 and 109.9)
  const bool dw_early = a.dx && (!p.few || int64_t(a.rows) * a.cols <= int64_t(1) << 24);
  for (int i = 0; i < p.pieces; ++i) {
    const int64_t v0 = i * p.piece, len = piece_len(p, a.rows, i);
    const uint8_t* w = a.w + v0 * a.ldw;
    const float* w_scale = a.w_scale + v0 / 128 * tile_cols;
    if (a.dx && !p.few)
      hw = {w, w_scale, nullptr, nullptr, tops + kPrepCtas, w16, back + 1, a.ldw, tile_cols, p.ldh, len, a.cols, prep_ctas,
            int(ctas_for(len * ((a.cols + 1023) / 1024), 8, half_ctas))};
    LossTile tile = {};
    if (hx.ctas + hw.ctas > 0) {
      tile.late = 1;
      launch_after(k_loss_half, unsigned(hx.ctas + hw.ctas), 256, 0, s, hx, hw);
      if (int rc = check("loss gradient (operands)")) return rc;
      hx.ctas = 0;
    }
    tile.end = kTileProbs, tile.zscale = a.scale, tile.lse = off;
    tile.target = target, tile.loss = a.loss, tile.first = int(v0);
    LinearArgs l{a.x, xs, w, w_scale, u, a.ldx, ld_xs, a.ldw, p.piece, a.n, int(len), a.cols, 0, status,
                 reinterpret_cast<float*>(base + p.scales), &tile};
    if (int rc = launch_linear_fp8(l, stream)) return rc;
    if (a.teacher) {
      FixArgs f{prep.y, off, a.logp, u, p.piece, a.ld_logp, a.n, int(v0), int(len)};
      launch_after(k_loss_fix, unsigned((a.n + 3) / 4), 128, 0, s, f);
      if (int rc = check("loss gradient (targets of a piece)")) return rc;
    }
    DxArgs gx = {};
    DwPieceArgs gw = {};
    unsigned dx_sums = 0, dw_sums = 0;
    if (a.dx && p.few) {
      auto* codes = reinterpret_cast<uint8_t*>(base + p.w);
      auto* scale = reinterpret_cast<float*>(base + p.dx);
      const int64_t lds = up_to(triple_rows(a.n), 4), ldc = up_to(len, 16);
      SplitArgs f{u, codes, scale, p.piece, ldc, lds, int(a.n), int(len)};
      launch_after(k_loss_split, unsigned((a.n * ((len + 127) / 128) + 7) / 8), 256, 0, s, f);
      if (int rc = check("loss gradient (few tokens)")) return rc;
      LossTile triples = {};
      triples.end = kTileTriples, triples.zscale = unscale, triples.lse = off, triples.factor = a.dloss;
      LinearArgs d{codes, scale, w, w_scale, a.dx, ldc, lds, a.ldw, a.ld_dx, triple_rows(a.n), int(len), a.cols, 1, status, nullptr, &triples};
      if (int rc = launch_linear_fp8(d, stream)) return rc;
    } else if (a.dx) {
      if (int rc = encode_map_codes(&tu, u, 2 * len, a.n, 2 * p.piece, 128)) return rc;
      if (int rc = encode_map_chunks(&tw, w16, a.cols, len, p.ldh, 2)) return rc;
      DxArgs& g = gx;
      g.part = reinterpret_cast<float*>(base + p.dx), g.row_factor = a.dloss, g.off = off, g.back = back + 1;
      g.out = static_cast<__nv_bfloat16*>(a.dx), g.factor = unscale, g.ldo = a.ld_dx;
      g.m = int(a.n), g.n = a.cols, g.k = int(len);
      g.add = i > 0, g.sh = p.dx_shares, g.status = status;
      void* args[] = {&tu, &tw, &g};
      const int pairs = std::min(cluster_slots()[2], g.sh.whole ? g.sh.tiles : g.sh.left() * g.sh.parts);
      if (int rc = launch_clusters("loss gradient (dx)", reinterpret_cast<const void*>(k_loss_dx), pairs, 2, PAIR_THREADS, DW_SMEM, args, s))
        return rc;
      if (i + 1 == p.pieces) dx_sums = unsigned(g.sh.tiles) * 16;
    }
    if (a.dw) {
      if (int rc = encode_map_chunks(&tu, u, len, a.n, p.piece, 2)) return rc;
      DwPieceArgs& g = gw;
      g.out = static_cast<__nv_bfloat16*>(a.dw) + v0 * a.ld_dw, g.ldo = a.ld_dw, g.m = int(len), g.n = a.cols, g.k = int(a.n);
      g.splits = dw_splits(a.n, len, a.cols);
      g.part = g.splits > 1 ? reinterpret_cast<float*>(base + p.dw) : nullptr;
      g.back = back, g.factor = unscale, g.accumulate = a.accumulate, g.late = dw_early;
      g.bytes = store_bytes(g.out, a.ld_dw, a.cols), g.status = status;
      to = tx;  // (not read by plain stores and shares)
      if (!g.part && g.bytes == 16)
        if (int rc = encode_map_bf16_out(&to, g.out, a.cols, len, a.ld_dw, 64)) return rc;
      const int64_t tiles = int64_t((g.m + PM - 1) / PM) * ((g.n + PN - 1) / PN);
      void* args[] = {&tu, &tx, &to, &g};
      if (int rc = launch_clusters("loss gradient (dw)", reinterpret_cast<const void*>(k_loss_dw),
                                   int(std::min<int64_t>(tiles * g.splits, cluster_slots()[2])), 2, PAIR_THREADS, DW_SMEM, args, s))
        return rc;
      if (g.part) dw_sums = unsigned(tiles * 16);
    }
    if (dx_sums + dw_sums > 0) {
      launch_after(k_loss_sums, dx_sums + dw_sums, 256, 0, s, gx, gw, int(dx_sums));
      if (int rc = check("loss gradient (sums)")) return rc;
    }
  }
  return BQ_OK;
}

}  // namespace bq
