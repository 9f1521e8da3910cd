// Host-side declarations of the fine-tuning operators' kernels (8-bit
// checkpoints and the gated activation, block norms, adapters).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nf4moe {

// Values held as bf16 or fp32 arrays, or as an 8-bit checkpoint.
enum Src { SRC_F32 = 0, SRC_BF16 = 1, SRC_MXINT8 = 2, SRC_MXFP8 = 3 };

hipError_t launch_ckpt8_quantize(int fmt, const void *x, bool x_bf16, int64_t n, uint8_t *codes, uint8_t *scale,
                                 hipStream_t s);
hipError_t launch_ckpt8_dequantize(int fmt, const uint8_t *codes, const uint8_t *scale, int64_t n, void *out,
                                   bool out_bf16, hipStream_t s);

struct GluArgs {
  int64_t R;
  int I;                     // I % 32 == 0
  int glu, inter;            // as GemmArgs
  float alpha, limit;
  const void *gu;            // [R, 2I]: bf16 / fp32 values, or 8-bit codes (backward)
  const uint8_t *gu_scale;   // 8-bit: e8m0 [R, 2I / 32]
  int src;                   // Src of gu
  // forward
  uint16_t *h;               // bf16 [R, I] (backward: optional)
  uint8_t *codes, *scale;    // optional 8-bit save of gu, format fmt
  int fmt;
  // backward
  const void *dh;            // [R, I] bf16 or fp32
  bool dh_bf16;
  const float *row_w;        // [R] or null
  uint16_t *dgu;             // bf16 [R, 2I]
  float *drow;               // [R] or null
};
hipError_t launch_glu_forward(const GluArgs &a, hipStream_t s);
hipError_t launch_glu_backward(const GluArgs &a, hipStream_t s);

// Post norm, gate, residual and the next pre norm of [T, H] rows.
struct NormArgs {
  int64_t T;
  int H;
  const void *x;             // residual stream, bf16 or fp32 (x_bf16)
  bool x_bf16;
  const uint16_t *f;         // block output, bf16, or null (x passes through)
  const float *w_post, *w_pre;   // [H] or null
  const void *gate;          // null, or by gate_kind
  int gate_kind;             // 0 none, 1 [H], 2 [T], 3 [T, H]
  bool gate_bf16;
  int gate_fn;               // 0 identity, 1 sigmoid, 2 tanh
  float alpha, eps;
  // forward
  void *x_new;               // as x
  uint16_t *y;               // bf16, or null without w_pre
  float *rstd_post, *rstd_pre;   // [T], written by the forward, read by the backward
  // backward (x is then the new stream that the forward wrote)
  const void *dx_new;        // as x, or null (zero)
  const uint16_t *dy;        // bf16 or null (no pre norm)
  void *dx;                  // as x
  uint16_t *df;              // bf16 or null
  float *dgate;              // fp32: [H], [T] or [T, H]
  float *dw_post, *dw_pre;   // [H]
  float *partial;            // [groups][2][H]
  int groups;
};
hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s);
int norm_backward_groups(int64_t T, int H);
constexpr int kNormMaxH = 16384;

// Adapters. Rows are grouped by adapter (stable, rows without one last) into
// tiles of up to 64 rows and chunks of up to adapter_chunk_rows(R) rows.
constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 128;
constexpr int kAdTile = 64;
constexpr int kMaxChunk = 2048;
struct AdapterPlan {
  int32_t *order;      // [R] row of each place in grouped order
  int32_t *counts;     // [0] tiles, [1] chunks
  int2 *chunks_of;     // [L] (chunks of the adapter, at least 1; first partial slot)
  int4 *tiles;         // (adapter or -1, first place, rows, 0)
  int4 *chunks;        // (adapter, first place, rows, partial slot or -1 when the adapter has one chunk)
  int32_t *hist;       // scratch
  int max_tiles, max_chunks, max_slots;
};
int adapter_chunk_rows(int R);
size_t adapter_plan_layout(int R, int L, void *base, AdapterPlan *p);   // bytes
// The plan (with ids), and the backward's turned weights: Bt [L, rank, N] and At [L,
// K, rank], each where given.
struct PrepareArgs {
  AdapterPlan plan;
  const int32_t *ids;  // or null: no plan to make
  int R, L, K, N, rank;
  const uint16_t *A, *B;
  uint16_t *At, *Bt;
};
hipError_t launch_adapter_prepare(const PrepareArgs &a, hipStream_t s);

// v[row][j] = sum_k x[row'][k] W1_l[j][k] for the rows of adapter l (W1 [L, rank, K]
// bf16), row' by row_of, and out[row][c] = base[row][c] + sum_j (m_l v[row][j])
// W2_l[c][j] (W2 [L, N, rank] bf16). low (optional): v, or m_l v with low_scaled, by
// row; zeros for rows without an adapter. m: scale [L] or null. The first launch makes
// v, the second out of it (out null: low alone, no second launch).
struct LowRankArgs {
  AdapterPlan plan;
  int R;
  const uint16_t *x;
  const int32_t *row_of;
  int x_rows;
  const uint16_t *W1, *W2;
  const float *scale;
  int K, N, rank;
  float *low;
  bool low_scaled;
  const void *base;    // or null: zeros
  void *out;
  bool bf16;           // base and out
  float *partial;      // scratch: [adapter_slices(R, K, rank)][R][rank]
  uint16_t *parts;     // scratch: adapter_parts_elems(max_tiles, rank) (null without out)
};
int adapter_slices(int R, int K, int rank);
size_t adapter_parts_elems(int tiles, int rank);
hipError_t launch_adapter_shrink(const LowRankArgs &a, hipStream_t s);
hipError_t launch_adapter_expand(const LowRankArgs &a, hipStream_t s);

// Per adapter l, out_l[j][c] (or [c][j], transposed) = m_l sum over the rows of l of
// p[row][j] v[row'][c]; a: v by src, b: v bf16. Each where out is given.
struct RowGradOne {
  const float *p;      // [R, rank]
  const void *v;       // [v_rows, C]
  const uint8_t *v_scale;
  const int32_t *row_of;
  int v_rows;
  const float *scale;
  int C;
  bool transposed;     // out [L, C, rank]
  float *out, *partial;   // partial: [max_slots][rank * C]
};
struct RowGradArgs {
  AdapterPlan plan;
  int R, L, rank, src;
  RowGradOne a, b;
  int merge;           // chunks of an adapter that a workgroup takes together (set by the launch)
};
hipError_t launch_adapter_rowgrad(const RowGradArgs &a, hipStream_t s);
hipError_t launch_fill_f32_zero(float *p, int64_t n, hipStream_t s);

// The forward of few rows in one launch, without a plan.
struct AdapterRowsArgs {
  const uint16_t *x;
  const int32_t *row_of, *ids;
  int x_rows, R, L, K, N, rank;
  const uint16_t *A, *B;
  const float *scale;
  const void *base;
  void *out;
  bool bf16;
  float *t;            // or null
};
bool adapter_rows_supported(int R, int K, int N, int rank);
hipError_t launch_adapter_rows(const AdapterRowsArgs &a, hipStream_t s);

}  // namespace nf4moe
