// Launchers of the layer operators (row_ops.cu, linear_fp8.cu).  Their callers
// (ops_api.cpp) have checked every argument; counts of zero never reach them
// unless said otherwise.
#pragma once

#include <cstddef>
#include <cstdint>

namespace bq {

struct EmbedArgs {
  const void* table;  // bf16 or E4M3
  const float* tscale;
  const void* ids;
  void* out;
  int64_t rows, ldt, n, ldo;
  float scale;
  int cols, kind, id_bits;
};
int launch_embed(const EmbedArgs& a, void* stream);

struct EmbedGradArgs {
  const void *dy, *ids;
  void* out;
  int64_t ld_dy, n, rows, ldo;
  float scale;
  int cols, id_bits, out_kind, accumulate;
};
size_t embed_grad_bytes(int64_t n, int64_t cols);
int launch_embed_grad(const EmbedGradArgs& a, void* ws, void* stream);  // n may be 0

struct RmsnormArgs {
  const void *x, *residual, *weight;
  void *h, *y;
  uint8_t* codes;
  float *code_scale, *rstd;
  int64_t ld_x, ld_r, ld_h, ld_y, ld_codes, ld_scale, n;
  float eps;
  int cols;
};
int launch_rmsnorm(const RmsnormArgs& a, void* stream);

struct RmsnormGradArgs {
  const void *dy, *h, *weight, *dh;
  const float* rstd;
  void *dx, *dw;
  int64_t ld_dy, ld_h, ld_dh, ld_dx, n;
  int cols, dw_kind, accumulate;
};
size_t rmsnorm_grad_bytes(int64_t n, int64_t cols);
int launch_rmsnorm_grad(const RmsnormGradArgs& a, void* ws, void* stream);  // n may be 0

// pad: the codes' rows may be written up to the next multiple of 8
int launch_quant_rows(const void* x, int64_t ldx, int64_t n, int cols, uint8_t* codes, int64_t ldc, float* scale,
                      int64_t lds, bool pad, void* stream);
// bf16 rows of X (from FP8 rows) and of dY (dy NULL: not wanted) at pitches ldo, ldyo
int launch_dw_inputs(const uint8_t* codes, int64_t ldc, const float* scale, int64_t lds, int64_t n, int cols, void* x_out,
                     int64_t ldo, const void* dy, int64_t ldy, int rows, void* dy_out, int64_t ldyo, void* stream);
// FP8 projections (linear_fp8.cu)
struct LinearArgs {
  const uint8_t* x;      // codes [n, red], pitch ldx (a multiple of 16)
  const float* x_scale;  // [ceil(red / 128)][ld_xs]
  const uint8_t* w;      // codes of the weight [rows, cols], pitch ldw (a multiple of 16)
  const float* w_scale;  // [ceil(rows / 128)][ceil(cols / 128)]
  void* out;             // bf16 [n, rows] (or [n, cols]: transposed weight)
  int64_t ldx, ld_xs, ldw, ldo, n;
  int rows, cols;
  int transposed;        // 0: out = x W^T (red = cols); 1: out = x W (red = rows)
  int* status;
  float* scale_ws;       // room for x_scale at a pitch of n + 3 at most (not used if x_scale is 16-byte
                         // aligned and ld_xs a multiple of 4)
};
int launch_linear_fp8(const LinearArgs& a, void* stream);

// D [rows, cols] (+)= dY^T X over n tokens, bf16 (linear_fp8.cu): dy [n, rows] with 16-byte
// aligned rows (padded: its pitch covers the next multiple of 64 columns), x [n, cols] with
// a pitch that does.  A product with too few tiles for the GPU is split over the tokens, its
// fp32 shares in part (dw_part_bytes).
struct DwArgs {
  const void *dy, *x;
  void* dw;
  float* part;
  int* status;
  int64_t ld_dy, ld_x, ld_dw, n;
  int rows, cols, padded, accumulate;
};
int dw_splits(int64_t n, int64_t rows, int64_t cols);
size_t dw_part_bytes(int splits, int64_t rows, int64_t cols);
int launch_dw(const DwArgs& a, void* stream);

// few tokens: the sum of outer products, straight from dy and the FP8 rows
bool dw_few(int64_t n, int64_t rows, int64_t cols);
int launch_dw_few(const void* dy, int64_t ld_dy, const uint8_t* codes, int64_t ldc, const float* scale, int64_t lds,
                  int n, int rows, int cols, void* dw, int64_t ld_dw, int accumulate, void* stream);

}  // namespace bq
