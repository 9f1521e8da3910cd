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
  float *partial;            // [groups][3][H]
  int groups;
};
hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s);
int norm_backward_groups(int64_t T, int H);
constexpr int kNormMaxH = 16384;

}  // namespace nf4moe
