// Host-side declarations of the dense operators' kernels (gated feed-forward, vocabulary
// loss and distillation, layer norm).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nf4moe {

// Up to so many rows a backward holds what it rounds between its products (dgu, P) as the sum of two bf16
// parts, the second in rows T .. 2 T - 1, and x twice. One row's largest value may be most of its
// gradients, and the rounding of it all of their error (up to 2^-8), and the products' tiles have the room.
// More rows have one part: a row's own roundings are then those of its largest values (in dx, and in the rows of dw
// that few others share), and what keeps them apart from row to row is that the values differ. So P leaves
// out the one factor that all rows of a mean loss have in common (HeadArgs::unit).
constexpr int kTwoParts = 64;
constexpr int kDenseMaxWidth = 1 << 20;   // H and I: 256 rows of it are below 2^31 bytes

// out[m][n] = sum_k X(m, k) Y(n, k) in bf16, or in fp32 to `part` by slices of K (added to what is
// there with `add`). X: element (m, k) at x[m * ldx + k], turned x[k * ldx + m]; Y turned:
// y[k * ldy + n]. `live`: a bit for each k, zero where Y's row k counts as zeros (turned X).
struct ProductArgs {
  const uint16_t *x, *y;
  int64_t ldx, ldy, M, N, K;
  uint16_t *out;        // [M, N], or null
  float *part;          // [slices][M][N]
  bool add;
  int slices;
  const uint64_t *live;
};
// The two products of a backward pass, both with y turned: `dx` with x as it lies, `dw` with x
// turned, together in one launch where both are given (K > 0). *unit (null: 1) is a factor of `out`; parts go without
// it, launch_join has it.
hipError_t launch_products(const ProductArgs *dx, const ProductArgs *dw, const float *unit, hipStream_t s);
// Slices of K, of `least` steps of 64 at least, that fill the card (alone) or half of it (beside a second
// product): of 8 for dx, of 12 for dw, which has two turned operands and more to join.
int product_slices(int64_t M, int64_t N, int64_t K, bool alone, int least);
// out bf16 [n] = the sum of the slices' parts, in order, times *unit (null: 1).
hipError_t launch_join(const float *part, int slices, int64_t n, const float *unit, uint16_t *out, hipStream_t s);

struct FfnArgs {
  int64_t T;
  int H, I, glu, inter;
  float alpha, limit;
  const uint16_t *x, *w13;   // [T, H], [2I, H]
  uint16_t *h;               // [T, I] (backward: optional)
  const uint16_t *dh;        // [T, I]
  uint16_t *dgu;             // [T, 2I] in w13's row order; up to kTwoParts rows: [2 T, 2I], in two parts
  uint16_t *x2;              // up to kTwoParts rows: [2 T, H], x twice (or null)
};
hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s);
hipError_t launch_ffn_dgu(const FfnArgs &a, hipStream_t s);

constexpr int kMaxTeacher = 1024;
// The vocabulary head: logits x W^T, by k_head_* kernels that never store them.
struct HeadArgs {
  int64_t T, V;
  int H, k;                  // k: teacher entries a row (0: labels)
  float tau;
  const uint16_t *x, *w;     // [T, H], [V, H]
  const int32_t *ids;        // [T] labels or [T, k]
  // forward
  const void *teacher;       // [T, k]
  bool teacher_bf16;
  float *loss, *lse;         // [T]
  float *q, *logits;         // [T, k]
  float2 *stats;             // [head_stat_chunks][T]: (maximum, sum) of a chunk of columns
  float *picked;             // [T] the label's logit
  // both: the teacher's entries of each 16 rows, sorted by their 128 columns (kHeadChunk)
  uint32_t *list;            // [T / 16][16 k]: j << 11 | row % 16 << 7 | id % 128
  int32_t *offsets;          // [T / 16][chunks + 1]
  // backward
  const float *dloss;        // [T]
  int64_t v0, vn, vp;        // the piece of the vocabulary, and the row stride of P
  uint16_t *P;               // [T, vp]; up to kTwoParts rows: [2 T, vp], in two parts
  uint16_t *x2;              // up to kTwoParts rows: [2 T, H], x twice, zeros in the rows that do not count (or null)
  uint64_t *live;            // [T / 64] or null: a bit for each row, set where it has a gradient (written with the first piece)
  // more than kTwoParts rows (or null): the factor that P leaves out and the products' outputs get, in fp32
  float *unit;
};
constexpr int kHeadChunk = 128;
int64_t head_stat_chunks(int64_t T, int64_t V, int H);
hipError_t launch_head_forward(const HeadArgs &a, hipStream_t s);
// What comes before a backward's pieces: the teacher's lists, and the unit.
hipError_t launch_head_prepare(const HeadArgs &a, hipStream_t s);
hipError_t launch_head_piece(const HeadArgs &a, hipStream_t s);
int64_t head_piece(int64_t rows, int64_t V);   // rows of P, one at least

struct LayerNormArgs {
  int64_t T;
  int H;
  bool x_bf16, y_bf16;
  const void *x;
  const float *w, *b;        // [H] or null
  float eps;
  void *y;                   // forward
  float *mean, *rstd;        // [T], written by the forward, read by the backward
  // backward
  const void *dy;            // as y
  const void *dx_base;       // as x, or null
  void *dx;                  // as x, or null
  float *dw, *db;            // [H] or null
  float *partial;            // [groups][2][H]
  int groups;
};
constexpr int kLayerNormMaxH = 16384;
hipError_t launch_layer_norm_forward(const LayerNormArgs &a, hipStream_t s);
hipError_t launch_layer_norm_backward(const LayerNormArgs &a, hipStream_t s);
int layer_norm_groups(int64_t T, int H);

}  // namespace nf4moe
