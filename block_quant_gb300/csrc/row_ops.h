// Launchers of the layer operators (row_ops.cu, linear_fp8.cu).  Their callers
// (ops_api.cpp) have checked every argument; counts of zero never reach them
// unless said otherwise.
#pragma once

#include <vector_types.h>

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
// What k_linear and k_linear_pair do with a tile of products: rows of out, or, for a loss
// (loss_fp8.cu), statistics of each row's part of the tile (and the logits of the row's listed words in
// it), its scaled probabilities, or the sum of three rows of products, a token's
enum TileEnd { kTileOut = 0, kTileStats = 1, kTileProbs = 2, kTileTriples = 3, kTilePicks = 4 };
constexpr int kPartCols = 64;  // of statistics
struct LossTile {
  int end;
  float zscale;      // a logit is zscale times the product
  // late (statistics, probabilities): the launch before neither writes what this one reads nor reads what it
  // writes, and has itself waited for all that came before: this one begins beside it and waits for its end at
  // its own
  int late;
  float2* stats;     // kTileStats: [part][ld_stats] and
  uint8_t* at;       // the largest logit's column in its part
  int64_t ld_stats;
  // kTilePicks (statistics too; not where k_linear splits a tile): records[w][t] (loss_tile.h; w to the number of parts)
  // of row t's listed words in part w, words[t][..], whose logits go to picked[t][..]
  const uint32_t* records;
  const uint16_t* words;
  float* picked;
  int64_t ld_records, ld_picked;
  int listed;        // pitch of words
  // kTileProbs: each row's log-sum, its class (-1: none) and loss, and the first word's number
  const float* lse;
  const int* target;
  const float* loss;
  int first;
  // kTileTriples (transposed): rows 3 i, 3 i + 1, 3 i + 2 of each 128 are token 42 j + i's, i < 42; each token's
  // factor beside zscale, lse as above
  const float* factor;
};

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
  LossTile* loss = nullptr;  // kTileProbs: out is fp16, 16-byte aligned, its pitch a multiple of 256 that covers the width
};
int launch_linear_fp8(const LinearArgs& a, void* stream);
bool linear_on_pairs(int64_t n, int64_t width, int64_t red);  // whether out = x W^T takes the CTA pairs
bool linear_whole_tiles(int64_t n, int64_t width, int64_t red);  // whether it takes one CTA or pair a tile
double linear_small_us(int64_t n, int64_t width, int64_t red);  // what out = x W costs without them
// X's scales [groups][ldx] at a pitch whose rows 16-byte copies can read
int launch_copy_scales(const float* x, int64_t ldx, int64_t n, int64_t groups, float* out, int64_t ldo, void* stream);

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

// Softmax losses over an FP8 head (loss_fp8.cu).  Targets of row t: pair i < k of ids (32 or 64
// bits, pitch ld_ids), with the teacher's logits (NULL: one pair of weight 1, a class).
struct LossArgs {
  const uint8_t* x;
  const float* x_scale;
  const uint8_t* w;
  const float* w_scale;
  const void *ids, *teacher;
  float *loss, *lse, *logp;  // forward: written; gradient: read (a class's logp is -loss)
  const float* dloss;
  void *dx, *dw;             // gradient, either may be NULL
  int64_t ldx, ld_xs, ldw, ld_ids, ld_teacher, ld_logp, ld_dx, ld_dw, n;
  float scale;
  int rows, cols, k, id_bits, teacher_kind, accumulate;
};
size_t loss_bytes(int64_t n, int64_t rows, int64_t cols);
size_t loss_grad_bytes(int64_t n, int64_t rows, int64_t cols);
int launch_loss(const LossArgs& a, void* ws, void* stream);
int launch_loss_grad(const LossArgs& a, void* ws, void* stream);

}  // namespace bq
