// C ABI of the layer operators: argument checks and dispatch to the kernels of
// row_ops.cu, linear_fp8.cu and ns_gemm.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "bq_internal.h"
#include "row_ops.h"

using namespace bq;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 27, kMaxCols = 65536, kMaxRows = int64_t(1) << 30;
constexpr size_t kStatusBytes = 256;  // device error word at the head of a projection's workspace

int fail(int code, const char* who, const char* what) { return set_error(code, std::string(who) + ": " + what); }

bool off(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

// a pitch that a matrix of at most one row never uses counts as its width
int64_t pitch(int64_t ld, int64_t n, int64_t width) { return n <= 1 ? std::max(ld, width) : ld; }

int check_sizes(const char* who, int64_t n, int64_t rows, int64_t cols) {
  if (n < 0 || n > kMaxTokens) return fail(BQ_EINVAL, who, "n outside [0, 2^27]");
  if (rows < 1 || rows > kMaxRows) return fail(BQ_EINVAL, who, "rows outside [1, 2^30]");
  if (cols < 1 || cols > kMaxCols) return fail(BQ_EINVAL, who, "cols outside [1, 65536]");
  return BQ_OK;
}

int check_ws(const char* who, const void* ws, size_t have, size_t need) {
  if (!ws) return fail(BQ_EINVAL, who, "NULL workspace");
  if (off(ws, 256)) return fail(BQ_EALIGN, who, "workspace must be 256-byte aligned");
  if (have < need) return fail(BQ_ENOSPC, who, "workspace too small");
  return BQ_OK;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t up64(int64_t x) { return (x + 63) / 64 * 64; }
int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

// forward: X's scales, where their own pitch does not serve; dx: codes and scales of
// dy; dw: bf16 rows of X and, where dy's own pitch does not serve, of dy, and the parts
// of a product split over the tokens
struct LinearWs {
  size_t codes, scales, x, dy, part, bytes;
};

int64_t up4(int64_t x) { return (x + 3) / 4 * 4; }

LinearWs linear_ws(int64_t n, int64_t rows, int64_t cols) {
  LinearWs p;
  p.codes = kStatusBytes;
  p.scales = p.codes + up(size_t(n) * size_t(up16(rows)));
  const size_t dx = p.scales + up(size_t((rows + 127) / 128) * size_t(up4(n)) * 4);
  const size_t fwd = kStatusBytes + up(size_t((cols + 127) / 128) * size_t(up4(n)) * 4);
  p.x = kStatusBytes;
  p.dy = p.x + up(size_t(n) * size_t(up64(cols)) * 2);
  p.part = p.dy + up(size_t(n) * size_t(up64(rows)) * 2);
  const size_t dw = p.part + dw_part_bytes(dw_splits(n, rows, cols), rows, cols);
  p.bytes = std::max({dx, dw, fwd});
  return p;
}

// tensor-core operands: rows of the product's summed index and tile counts as ints
int check_linear(const char* who, int64_t n, int64_t rows, int64_t cols) {
  if (int rc = check_sizes(who, n, rows, cols)) return rc;
  if (rows > (int64_t(1) << 24)) return fail(BQ_EINVAL, who, "rows above 2^24");
  if (cols % 16) return fail(BQ_EALIGN, who, "cols must be a multiple of 16");
  return BQ_OK;
}

int check_weight(const char* who, const uint8_t* w, int64_t ldw, const float* w_scale, int64_t cols) {
  if (!w || !w_scale) return fail(BQ_EINVAL, who, "NULL weight");
  if (ldw < cols) return fail(BQ_EINVAL, who, "weight pitch below cols");
  if (off(w, 16) || ldw % 16 || off(w_scale, 4))
    return fail(BQ_EALIGN, who, "weight codes 16-byte aligned with a pitch multiple of 16, scales 4-byte aligned");
  return BQ_OK;
}

}  // namespace

extern "C" {

int bq_embed(const void* table, int kind, const float* table_scale, int64_t rows, int64_t cols, int64_t ld_table,
             const void* ids, int id_bits, int64_t n, float scale, void* out, int64_t ld_out, bq_stream_t stream) {
  const char* who = "bq_embed";
  if (int rc = check_sizes(who, n, rows, cols)) return rc;
  if (kind != BQ_ROWS_BF16 && kind != BQ_ROWS_FP8) return fail(BQ_EINVAL, who, "table kind must be bf16 or FP8");
  if (id_bits != 32 && id_bits != 64) return fail(BQ_EINVAL, who, "id_bits must be 32 or 64");
  if (n == 0) return BQ_OK;
  if (!table || !ids || !out || (kind == BQ_ROWS_FP8 && !table_scale)) return fail(BQ_EINVAL, who, "NULL argument");
  ld_table = pitch(ld_table, rows, cols), ld_out = pitch(ld_out, n, cols);
  if (ld_table < cols || ld_out < cols) return fail(BQ_EINVAL, who, "pitch below cols");
  if ((kind == BQ_ROWS_BF16 && off(table, 2)) || off(out, 2) || off(ids, uintptr_t(id_bits / 8)) || off(table_scale, 4))
    return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  return launch_embed(EmbedArgs{table, table_scale, ids, out, rows, ld_table, n, ld_out, scale, int(cols), kind, id_bits},
                      stream);
}

int bq_embed_grad_workspace(int64_t n, int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(BQ_EINVAL, "bq_embed_grad_workspace", "NULL argument");
  if (int rc = check_sizes("bq_embed_grad_workspace", n, rows, cols)) return rc;
  *bytes = embed_grad_bytes(n, cols);
  return BQ_OK;
}

int bq_embed_grad(const void* dy, int64_t ld_dy, const void* ids, int id_bits, int64_t n, float scale, int64_t rows,
                  int64_t cols, void* out, int out_kind, int64_t ld_out, int accumulate, void* ws, size_t ws_bytes,
                  bq_stream_t stream) {
  const char* who = "bq_embed_grad";
  if (int rc = check_sizes(who, n, rows, cols)) return rc;
  if (out_kind != BQ_ROWS_BF16 && out_kind != BQ_ROWS_FP32) return fail(BQ_EINVAL, who, "out kind must be bf16 or fp32");
  if (id_bits != 32 && id_bits != 64) return fail(BQ_EINVAL, who, "id_bits must be 32 or 64");
  if (!out || (n > 0 && (!dy || !ids))) return fail(BQ_EINVAL, who, "NULL argument");
  ld_dy = pitch(ld_dy, n, cols), ld_out = pitch(ld_out, rows, cols);
  if (ld_dy < cols || ld_out < cols) return fail(BQ_EINVAL, who, "pitch below cols");
  if (off(dy, 2) || off(out, out_kind == BQ_ROWS_FP32 ? 4 : 2) || off(ids, uintptr_t(id_bits / 8)))
    return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  if (int rc = check_ws(who, ws, ws_bytes, embed_grad_bytes(n, cols))) return rc;
  if (n == 0 && accumulate) return BQ_OK;
  return launch_embed_grad(EmbedGradArgs{dy, ids, out, ld_dy, n, rows, ld_out, scale, int(cols), id_bits, out_kind,
                                         accumulate ? 1 : 0},
                           ws, stream);
}

int bq_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight, float eps,
               int64_t n, int64_t cols, void* h, int64_t ld_h, void* y, int64_t ld_y, uint8_t* codes, int64_t ld_codes,
               float* code_scale, int64_t ld_scale, float* rstd, bq_stream_t stream) {
  const char* who = "bq_rmsnorm";
  if (int rc = check_sizes(who, n, 1, cols)) return rc;
  if (!(eps >= 0.f)) return fail(BQ_EINVAL, who, "eps must not be negative or NaN");
  if (n == 0) return BQ_OK;
  if (!x || !weight || (residual && !h) || (codes && !code_scale)) return fail(BQ_EINVAL, who, "NULL argument");
  if (!h && !y && !codes && !rstd) return fail(BQ_EINVAL, who, "no output");
  if (!residual) h = nullptr;
  ld_x = pitch(ld_x, n, cols), ld_residual = pitch(ld_residual, n, cols), ld_h = pitch(ld_h, n, cols);
  ld_y = pitch(ld_y, n, cols), ld_codes = pitch(ld_codes, n, cols), ld_scale = pitch(ld_scale, cols <= 128 ? 1 : 2, n);
  if (ld_x < cols || (residual && ld_residual < cols) || (h && ld_h < cols) || (y && ld_y < cols) ||
      (codes && (ld_codes < cols || ld_scale < n)))
    return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(x, 2) || off(residual, 2) || off(weight, 2) || off(h, 2) || off(y, 2) || off(code_scale, 4) || off(rstd, 4))
    return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  return launch_rmsnorm(RmsnormArgs{x, residual, weight, h, y, codes, code_scale, rstd, ld_x, ld_residual, ld_h, ld_y,
                                    ld_codes, ld_scale, n, eps, int(cols)},
                        stream);
}

int bq_rmsnorm_grad_workspace(int64_t n, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(BQ_EINVAL, "bq_rmsnorm_grad_workspace", "NULL argument");
  if (int rc = check_sizes("bq_rmsnorm_grad_workspace", n, 1, cols)) return rc;
  *bytes = rmsnorm_grad_bytes(n, cols);
  return BQ_OK;
}

int bq_rmsnorm_grad(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* weight, const float* rstd,
                    const void* dh, int64_t ld_dh, int64_t n, int64_t cols, void* dx, int64_t ld_dx, void* dw,
                    int dw_kind, int accumulate, void* ws, size_t ws_bytes, bq_stream_t stream) {
  const char* who = "bq_rmsnorm_grad";
  if (int rc = check_sizes(who, n, 1, cols)) return rc;
  if (dw_kind != BQ_ROWS_BF16 && dw_kind != BQ_ROWS_FP32) return fail(BQ_EINVAL, who, "dw kind must be bf16 or fp32");
  if (!weight || !dw || (n > 0 && (!dy || !h || !rstd || !dx))) return fail(BQ_EINVAL, who, "NULL argument");
  ld_dy = pitch(ld_dy, n, cols), ld_h = pitch(ld_h, n, cols), ld_dh = pitch(ld_dh, n, cols);
  ld_dx = pitch(ld_dx, n, cols);
  if (ld_dy < cols || ld_h < cols || (dh && ld_dh < cols) || ld_dx < cols)
    return fail(BQ_EINVAL, who, "pitch below cols");
  if (off(dy, 2) || off(h, 2) || off(weight, 2) || off(rstd, 4) || off(dh, 2) || off(dx, 2) ||
      off(dw, dw_kind == BQ_ROWS_FP32 ? 4 : 2))
    return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  if (int rc = check_ws(who, ws, ws_bytes, rmsnorm_grad_bytes(n, cols))) return rc;
  if (n == 0 && accumulate) return BQ_OK;
  return launch_rmsnorm_grad(RmsnormGradArgs{dy, h, weight, dh, rstd, dx, dw, ld_dy, ld_h, ld_dh, ld_dx, n, int(cols),
                                             dw_kind, accumulate ? 1 : 0},
                             ws, stream);
}

int bq_quant_rows_fp8(const void* x, int64_t ld_x, int64_t n, int64_t cols, uint8_t* codes, int64_t ld_codes,
                      float* code_scale, int64_t ld_scale, bq_stream_t stream) {
  const char* who = "bq_quant_rows_fp8";
  if (int rc = check_sizes(who, n, 1, cols)) return rc;
  if (n == 0) return BQ_OK;
  if (!x || !codes || !code_scale) return fail(BQ_EINVAL, who, "NULL argument");
  ld_x = pitch(ld_x, n, cols), ld_codes = pitch(ld_codes, n, cols);
  ld_scale = pitch(ld_scale, cols <= 128 ? 1 : 2, n);
  if (ld_x < cols || ld_codes < cols || ld_scale < n) return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(x, 2) || off(code_scale, 4)) return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  return launch_quant_rows(x, ld_x, n, int(cols), codes, ld_codes, code_scale, ld_scale, false, stream);
}

int bq_linear_fp8_workspace(int64_t n, int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(BQ_EINVAL, "bq_linear_fp8_workspace", "NULL argument");
  if (int rc = check_linear("bq_linear_fp8_workspace", n, rows, cols)) return rc;
  *bytes = linear_ws(n, rows, cols).bytes;
  return BQ_OK;
}

int bq_linear_fp8(const uint8_t* x, int64_t ld_x, const float* x_scale, int64_t ld_scale, const uint8_t* w,
                  int64_t ld_w, const float* w_scale, int64_t n, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                  void* ws, size_t ws_bytes, bq_stream_t stream) {
  const char* who = "bq_linear_fp8";
  if (int rc = check_linear(who, n, rows, cols)) return rc;
  if (int rc = check_ws(who, ws, ws_bytes, linear_ws(n, rows, cols).bytes)) return rc;
  if (n == 0) return BQ_OK;
  ld_x = n == 1 ? std::max(up16(ld_x), cols) : ld_x;
  ld_out = pitch(ld_out, n, rows), ld_scale = pitch(ld_scale, cols <= 128 ? 1 : 2, n);
  ld_w = rows == 1 ? std::max(up16(ld_w), cols) : ld_w;
  if (int rc = check_weight(who, w, ld_w, w_scale, cols)) return rc;
  if (!x || !x_scale || !out) return fail(BQ_EINVAL, who, "NULL argument");
  if (ld_x < cols || ld_out < rows || ld_scale < n) return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(x, 16) || ld_x % 16) return fail(BQ_EALIGN, who, "codes must be 16-byte aligned with a pitch multiple of 16");
  if (off(x_scale, 4) || off(out, 2)) return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  return launch_linear_fp8(LinearArgs{x, x_scale, w, w_scale, out, ld_x, ld_scale, ld_w, ld_out, n, int(rows), int(cols),
                                      0, static_cast<int*>(ws),
                                      reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kStatusBytes)},
                           stream);
}

int bq_linear_fp8_dx(const void* dy, int64_t ld_dy, const uint8_t* w, int64_t ld_w, const float* w_scale, int64_t n,
                     int64_t rows, int64_t cols, void* dx, int64_t ld_dx, void* ws, size_t ws_bytes,
                     bq_stream_t stream) {
  const char* who = "bq_linear_fp8_dx";
  if (int rc = check_linear(who, n, rows, cols)) return rc;
  const LinearWs p = linear_ws(n, rows, cols);
  if (int rc = check_ws(who, ws, ws_bytes, p.bytes)) return rc;
  if (n == 0) return BQ_OK;
  ld_dy = pitch(ld_dy, n, rows), ld_dx = pitch(ld_dx, n, cols);
  ld_w = rows == 1 ? std::max(up16(ld_w), cols) : ld_w;
  if (int rc = check_weight(who, w, ld_w, w_scale, cols)) return rc;
  if (!dy || !dx) return fail(BQ_EINVAL, who, "NULL argument");
  if (ld_dy < rows || ld_dx < cols) return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(dy, 2) || off(dx, 2)) return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  auto* base = static_cast<unsigned char*>(ws);
  auto* codes = base + p.codes;
  auto* scales = reinterpret_cast<float*>(base + p.scales);
  const int64_t ldc = up16(rows), lds = up4(n);
  if (int rc = launch_quant_rows(dy, ld_dy, n, int(rows), codes, ldc, scales, lds, true, stream)) return rc;
  return launch_linear_fp8(LinearArgs{codes, scales, w, w_scale, dx, ldc, lds, ld_w, ld_dx, n, int(rows), int(cols), 1,
                                      static_cast<int*>(ws), nullptr},
                           stream);
}

int bq_linear_fp8_dw(const void* dy, int64_t ld_dy, const uint8_t* x, int64_t ld_x, const float* x_scale,
                     int64_t ld_scale, int64_t n, int64_t rows, int64_t cols, void* dw, int64_t ld_dw, int accumulate,
                     void* ws, size_t ws_bytes, bq_stream_t stream) {
  const char* who = "bq_linear_fp8_dw";
  if (int rc = check_linear(who, n, rows, cols)) return rc;
  const LinearWs p = linear_ws(n, rows, cols);
  if (int rc = check_ws(who, ws, ws_bytes, p.bytes)) return rc;
  ld_dw = pitch(ld_dw, rows, cols);
  if (!dw) return fail(BQ_EINVAL, who, "NULL argument");
  if (ld_dw < cols) return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(dw, 2)) return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  if (n == 0) {
    if (accumulate) return BQ_OK;
    const cudaError_t e = cudaMemset2DAsync(dw, size_t(ld_dw) * 2, 0, size_t(cols) * 2, size_t(rows),
                                            reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BQ_OK : fail(BQ_ECUDA, who, cudaGetErrorString(e));
  }
  ld_dy = pitch(ld_dy, n, rows), ld_scale = pitch(ld_scale, cols <= 128 ? 1 : 2, n);
  ld_x = n == 1 ? std::max(up16(ld_x), cols) : ld_x;
  if (!dy || !x || !x_scale) return fail(BQ_EINVAL, who, "NULL argument");
  if (ld_dy < rows || ld_x < cols || ld_scale < n) return fail(BQ_EINVAL, who, "pitch below the width");
  if (off(x, 16) || ld_x % 16) return fail(BQ_EALIGN, who, "codes must be 16-byte aligned with a pitch multiple of 16");
  if (off(dy, 2) || off(x_scale, 4)) return fail(BQ_EALIGN, who, "pointer not aligned to its element type");
  auto* base = static_cast<unsigned char*>(ws);
  const int64_t ldxb = up64(cols);
  if (dw_few(n, rows, cols))
    return launch_dw_few(dy, ld_dy, x, ld_x, x_scale, ld_scale, int(n), int(rows), int(cols), dw, ld_dw,
                         accumulate ? 1 : 0, stream);
  // dy as it stands where its rows are 16-byte aligned, as the product's copies want them
  const bool copy = off(dy, 16) || ld_dy % 8;
  const int64_t lda = copy ? up64(rows) : ld_dy;
  if (int rc = launch_dw_inputs(x, ld_x, x_scale, ld_scale, n, int(cols), base + p.x, ldxb, copy ? dy : nullptr, ld_dy,
                                int(rows), base + p.dy, lda, stream))
    return rc;
  return launch_dw(DwArgs{copy ? base + p.dy : dy, base + p.x, dw, reinterpret_cast<float*>(base + p.part),
                          static_cast<int*>(ws), lda, ldxb, ld_dw, n, int(rows), int(cols), copy || rows % 64 == 0,
                          accumulate ? 1 : 0},
                   stream);
}

int bq_linear_check(void* ws, size_t ws_bytes, bq_stream_t stream) {
  if (!ws || ws_bytes < kStatusBytes) return fail(BQ_EINVAL, "bq_linear_check", "bad workspace");
  int status = 0;
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaMemcpy(&status, ws, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && status) e = cudaMemset(ws, 0, sizeof(int));
  if (e != cudaSuccess) return fail(BQ_ECUDA, "bq_linear_check", cudaGetErrorString(e));
  if (status) return set_error(BQ_ECUDA, "bq_linear_fp8: a device wait timed out (site " + std::to_string(status) + ")");
  return BQ_OK;
}

int bq_call(int op, const void* args) {
  if (!args) return fail(BQ_EINVAL, "bq_call", "NULL argument");
  const unsigned char* at = static_cast<const unsigned char*>(args);
  auto q = [&](int i) {
    int64_t v;
    std::memcpy(&v, at + 8 * i, 8);
    return v;
  };
  auto f = [&](int i) {
    double v;
    std::memcpy(&v, at + 8 * i, 8);
    return float(v);
  };
  auto p = [&](int i) { return reinterpret_cast<void*>(intptr_t(q(i))); };
  auto b = [&](int i) { return static_cast<uint8_t*>(p(i)); };
  auto s = [&](int i) { return static_cast<float*>(p(i)); };
  auto st = [&](int i) { return static_cast<bq_stream_t>(p(i)); };
  switch (op) {
    case BQ_CALL_EMBED:
      return bq_embed(p(0), int(q(1)), s(2), q(3), q(4), q(5), p(6), int(q(7)), q(8), f(9), p(10), q(11), st(12));
    case BQ_CALL_EMBED_GRAD:
      return bq_embed_grad(p(0), q(1), p(2), int(q(3)), q(4), f(5), q(6), q(7), p(8), int(q(9)), q(10), int(q(11)),
                           p(12), size_t(q(13)), st(14));
    case BQ_CALL_RMSNORM:
      return bq_rmsnorm(p(0), q(1), p(2), q(3), p(4), f(5), q(6), q(7), p(8), q(9), p(10), q(11), b(12), q(13), s(14),
                        q(15), s(16), st(17));
    case BQ_CALL_RMSNORM_GRAD:
      return bq_rmsnorm_grad(p(0), q(1), p(2), q(3), p(4), s(5), p(6), q(7), q(8), q(9), p(10), q(11), p(12),
                             int(q(13)), int(q(14)), p(15), size_t(q(16)), st(17));
    case BQ_CALL_QUANT_ROWS:
      return bq_quant_rows_fp8(p(0), q(1), q(2), q(3), b(4), q(5), s(6), q(7), st(8));
    case BQ_CALL_LINEAR:
      return bq_linear_fp8(b(0), q(1), s(2), q(3), b(4), q(5), s(6), q(7), q(8), q(9), p(10), q(11), p(12),
                           size_t(q(13)), st(14));
    case BQ_CALL_LINEAR_DX:
      return bq_linear_fp8_dx(p(0), q(1), b(2), q(3), s(4), q(5), q(6), q(7), p(8), q(9), p(10), size_t(q(11)), st(12));
    case BQ_CALL_LINEAR_DW:
      return bq_linear_fp8_dw(p(0), q(1), b(2), q(3), s(4), q(5), q(6), q(7), q(8), p(9), q(10), int(q(11)), p(12),
                              size_t(q(13)), st(14));
    default: return fail(BQ_EINVAL, "bq_call", "unknown call");
  }
}

}  // extern "C"
