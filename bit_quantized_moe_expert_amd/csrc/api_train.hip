// C ABI of the fine-tuning operators (declared in include/nf4moe.h): host-side
// validation, workspace carving and launches. Every check runs before anything
// is enqueued; on a non-OK status nothing was launched.
#include <math.h>

#include "../../include/nf4moe.h"
#include "ckpt8.h"
#include "internal.h"
#include "status.h"
#include "train.h"

using namespace nf4moe;

namespace {

bool dt_ok(int dt) { return dt == NF4MOE_DT_F32 || dt == NF4MOE_DT_BF16; }
size_t dt_bytes(int dt) { return dt == NF4MOE_DT_BF16 ? 2 : 4; }
bool ck_ok(int f) { return f == NF4MOE_CKPT_MXINT8 || f == NF4MOE_CKPT_MXFP8; }

nf4moe_status_t check_ckpt8(int32_t fmt, const void *dense, nf4moe_dtype_t dt, int64_t rows, int64_t K,
                            const void *codes, const void *scale) {
  if (!ck_ok(fmt)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown checkpoint format %d", (int)fmt);
  if (!dt_ok(dt)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (rows < 0) return fail(NF4MOE_ERR_INVALID_ARG, "rows=%lld < 0", (long long)rows);
  if (K <= 0 || K % 32) return fail(NF4MOE_ERR_INVALID_ARG, "K=%lld must be a positive multiple of 32", (long long)K);
  if (rows > ((int64_t)1 << 46) / K) return fail(NF4MOE_ERR_UNSUPPORTED, "rows * K too large");
  if (rows == 0) return NF4MOE_OK;
  if (!dense || !codes || !scale) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(dense, dt_bytes(dt))) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  return NF4MOE_OK;
}

// What both directions of the gated activation ask of their arguments.
nf4moe_status_t check_glu(int64_t R, int32_t I, int32_t glu, float alpha, float limit, int32_t inter) {
  if (R < 0) return fail(NF4MOE_ERR_INVALID_ARG, "R=%lld < 0", (long long)R);
  if (I <= 0 || I % 32) return fail(NF4MOE_ERR_INVALID_ARG, "I=%d must be a positive multiple of 32", I);
  if (R > ((int64_t)1 << 36) / I) return fail(NF4MOE_ERR_UNSUPPORTED, "R * I too large");
  if (glu != NF4MOE_GLU_SWIGLU && glu != NF4MOE_GLU_CLAMPED) return fail(NF4MOE_ERR_INVALID_ARG, "unknown glu %d", glu);
  if (glu == NF4MOE_GLU_CLAMPED && !(alpha > 0.0f && alpha < 1e30f && limit > 0.0f && limit < 1e30f))
    return fail(NF4MOE_ERR_INVALID_ARG, "clamped GLU needs finite alpha > 0 and limit > 0");
  if (inter != 0 && inter != 1) return fail(NF4MOE_ERR_INVALID_ARG, "glu_interleaved must be 0 or 1");
  return NF4MOE_OK;
}

// What both directions of the block norm ask of their arguments.
nf4moe_status_t check_norm(const nf4moe_block_norm_t *n, int64_t T) {
  if (!n) return fail(NF4MOE_ERR_INVALID_ARG, "norm is NULL");
  if (T < 0 || T > 0x7fffffff) return fail(NF4MOE_ERR_INVALID_ARG, "T=%lld outside 0..2^31-1", (long long)T);
  if (n->H < 1 || n->H > kNormMaxH) return fail(NF4MOE_ERR_INVALID_ARG, "H=%d outside 1..%d", n->H, kNormMaxH);
  if (!dt_ok(n->x_dtype) || !dt_ok(n->gate_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype");
  if (n->gate_kind < NF4MOE_GATE_NONE || n->gate_kind > NF4MOE_GATE_FULL)
    return fail(NF4MOE_ERR_INVALID_ARG, "unknown gate kind %d", n->gate_kind);
  if (n->gate_fn < NF4MOE_GATE_IDENTITY || n->gate_fn > NF4MOE_GATE_TANH)
    return fail(NF4MOE_ERR_INVALID_ARG, "unknown gate function %d", n->gate_fn);
  if ((n->gate_kind != NF4MOE_GATE_NONE) != (n->gate != nullptr) && T > 0)
    return fail(NF4MOE_ERR_INVALID_ARG, "gate and gate_kind go together");
  if (!(n->eps >= 0.0f && n->eps < 1e30f) || !(fabsf(n->alpha) < 1e30f))
    return fail(NF4MOE_ERR_INVALID_ARG, "eps must be finite and >= 0, alpha finite");
  if (!aligned(n->w_post, 4) || !aligned(n->w_pre, 4) || !aligned(n->gate, dt_bytes(n->gate_dtype)))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  return NF4MOE_OK;
}

NormArgs norm_args(const nf4moe_block_norm_t &n, int64_t T) {
  NormArgs a = {};
  a.T = T, a.H = n.H, a.x_bf16 = n.x_dtype == NF4MOE_DT_BF16;
  a.w_post = n.w_post, a.w_pre = n.w_pre;
  a.gate = n.gate, a.gate_kind = n.gate_kind, a.gate_bf16 = n.gate_dtype == NF4MOE_DT_BF16, a.gate_fn = n.gate_fn;
  a.alpha = n.alpha, a.eps = n.eps;
  return a;
}

}  // namespace

extern "C" {

nf4moe_status_t nf4moe_ckpt8_quantize(nf4moe_ckpt8_t fmt, const void *x, nf4moe_dtype_t x_dtype, int64_t rows, int64_t K,
                                      uint8_t *codes, uint8_t *scale, void *stream) {
  const nf4moe_status_t st = check_ckpt8(fmt, x, x_dtype, rows, K, codes, scale);
  if (st != NF4MOE_OK || rows == 0) return st;
  return hip_status(launch_ckpt8_quantize(fmt, x, x_dtype == NF4MOE_DT_BF16, rows * K, codes, scale, (hipStream_t)stream),
                    "checkpoint quantize launch");
}

nf4moe_status_t nf4moe_ckpt8_dequantize(nf4moe_ckpt8_t fmt, const uint8_t *codes, const uint8_t *scale, int64_t rows,
                                        int64_t K, void *out, nf4moe_dtype_t out_dtype, void *stream) {
  const nf4moe_status_t st = check_ckpt8(fmt, out, out_dtype, rows, K, codes, scale);
  if (st != NF4MOE_OK || rows == 0) return st;
  return hip_status(launch_ckpt8_dequantize(fmt, codes, scale, rows * K, out, out_dtype == NF4MOE_DT_BF16, (hipStream_t)stream),
                    "checkpoint dequantize launch");
}

nf4moe_status_t nf4moe_glu_forward(const void *gu, nf4moe_dtype_t gu_dtype, int64_t R, int32_t I, int32_t glu,
                                   float glu_alpha, float glu_limit, int32_t glu_interleaved, uint16_t *h,
                                   nf4moe_ckpt8_t ckpt, uint8_t *codes, uint8_t *scale, void *stream) {
  const nf4moe_status_t st = check_glu(R, I, glu, glu_alpha, glu_limit, glu_interleaved);
  if (st != NF4MOE_OK) return st;
  if (!dt_ok(gu_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)gu_dtype);
  if ((codes == nullptr) != (scale == nullptr)) return fail(NF4MOE_ERR_INVALID_ARG, "codes and scale go together");
  if (codes && !ck_ok(ckpt)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown checkpoint format %d", (int)ckpt);
  if (R == 0) return NF4MOE_OK;
  if (!gu || !h) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(gu, dt_bytes(gu_dtype)) || !aligned(h, 2)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  GluArgs a = {};
  a.R = R, a.I = I, a.glu = glu, a.inter = glu_interleaved, a.alpha = glu_alpha, a.limit = glu_limit;
  a.gu = gu, a.src = gu_dtype == NF4MOE_DT_BF16 ? SRC_BF16 : SRC_F32;
  a.h = h, a.codes = codes, a.scale = scale, a.fmt = ckpt;
  return hip_status(launch_glu_forward(a, (hipStream_t)stream), "GLU launch");
}

nf4moe_status_t nf4moe_glu_backward(const void *dh, nf4moe_dtype_t dh_dtype, nf4moe_src_t gu_src, const void *gu,
                                    const uint8_t *gu_scale, int64_t R, int32_t I, int32_t glu, float glu_alpha,
                                    float glu_limit, int32_t glu_interleaved, const float *row_w, uint16_t *dgu,
                                    uint16_t *h, float *drow_w, void *stream) {
  const nf4moe_status_t st = check_glu(R, I, glu, glu_alpha, glu_limit, glu_interleaved);
  if (st != NF4MOE_OK) return st;
  if (!dt_ok(dh_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dh_dtype);
  if (gu_src < NF4MOE_SRC_F32 || gu_src > NF4MOE_SRC_MXFP8) return fail(NF4MOE_ERR_INVALID_ARG, "unknown source %d", (int)gu_src);
  if (R == 0) return NF4MOE_OK;
  const bool held = gu_src >= NF4MOE_SRC_MXINT8;
  if (!dh || !gu || !dgu || (held && !gu_scale)) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(dh, dt_bytes(dh_dtype)) || !aligned(gu, held ? 1 : gu_src == NF4MOE_SRC_F32 ? 4 : 2) || !aligned(dgu, 2) ||
      !aligned(h, 2) || !aligned(row_w, 4) || !aligned(drow_w, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  GluArgs a = {};
  a.R = R, a.I = I, a.glu = glu, a.inter = glu_interleaved, a.alpha = glu_alpha, a.limit = glu_limit;
  a.gu = gu, a.gu_scale = gu_scale, a.src = gu_src;
  a.dh = dh, a.dh_bf16 = dh_dtype == NF4MOE_DT_BF16, a.row_w = row_w;
  a.dgu = dgu, a.h = h, a.drow = drow_w;
  return hip_status(launch_glu_backward(a, (hipStream_t)stream), "GLU backward launch");
}

nf4moe_status_t nf4moe_block_norm_forward(const nf4moe_block_norm_t *norm, const void *x, const uint16_t *f, int64_t T,
                                          void *x_new, uint16_t *y, float *rstd_post, float *rstd_pre, void *stream) {
  const nf4moe_status_t st = check_norm(norm, T);
  if (st != NF4MOE_OK) return st;
  const nf4moe_block_norm_t &n = *norm;
  if (T > 0 && !f && (n.w_post || n.gate_kind != NF4MOE_GATE_NONE))  // an empty f may have no address
    return fail(NF4MOE_ERR_INVALID_ARG, "w_post and the gate need a block output f");
  if (T > 0 && !f && !n.w_pre) return fail(NF4MOE_ERR_INVALID_ARG, "neither a block output nor a pre norm: nothing to do");
  if (T == 0) return NF4MOE_OK;
  if (!x || (f && !x_new) || (n.w_pre && (!y || !rstd_pre)) || (n.w_post && !rstd_post))
    return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, dt_bytes(n.x_dtype)) || !aligned(x_new, dt_bytes(n.x_dtype)) || !aligned(f, 2) || !aligned(y, 2) ||
      !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  NormArgs a = norm_args(n, T);
  a.x = x, a.f = f, a.x_new = x_new, a.y = y, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
  return hip_status(launch_norm_forward(a, (hipStream_t)stream), "norm launch");
}

size_t nf4moe_block_norm_workspace_bytes(int32_t H, int64_t T) {
  if (H < 1 || H > kNormMaxH || T < 1 || T > 0x7fffffff) return 0;
  return align_up((size_t)norm_backward_groups(T, H) * 3 * H * sizeof(float));
}

nf4moe_status_t nf4moe_block_norm_backward(const nf4moe_block_norm_t *norm, const void *dx_new, const uint16_t *dy,
                                           const void *x_new, const uint16_t *f, const float *rstd_post,
                                           const float *rstd_pre, int64_t T, void *dx, uint16_t *df, float *dgate,
                                           float *dw_post, float *dw_pre, void *ws, size_t ws_bytes, void *stream) {
  const nf4moe_status_t st = check_norm(norm, T);
  if (st != NF4MOE_OK) return st;
  const nf4moe_block_norm_t &n = *norm;
  if (T > 0 && !f && (n.w_post || n.gate_kind != NF4MOE_GATE_NONE))  // an empty f may have no address
    return fail(NF4MOE_ERR_INVALID_ARG, "w_post and the gate need a block output f");
  if (T > 0 && !f && !n.w_pre) return fail(NF4MOE_ERR_INVALID_ARG, "neither a block output nor a pre norm: nothing to do");
  const size_t gn = n.gate_kind == NF4MOE_GATE_CHANNEL ? (size_t)n.H : 0;
  hipStream_t s = (hipStream_t)stream;
  if ((n.w_pre && !dw_pre) || (n.w_post && !dw_post) || (gn && !dgate))
    return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(dw_pre, 4) || !aligned(dw_post, 4) || !aligned(dgate, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (T == 0) {  // the sums over no rows
    hipError_t e = hipSuccess;
    if (n.w_pre) e = launch_fill_i32((int32_t *)dw_pre, n.H, 0, s);
    if (e == hipSuccess && n.w_post) e = launch_fill_i32((int32_t *)dw_post, n.H, 0, s);
    if (e == hipSuccess && gn) e = launch_fill_i32((int32_t *)dgate, n.H, 0, s);
    return hip_status(e, "fill");
  }
  if (!dx || (f && !df) || (n.gate_kind != NF4MOE_GATE_NONE && !dgate) || (!dx_new && !n.w_pre) ||
      (n.w_pre && (!dy || !x_new || !rstd_pre)) || (n.w_post && !rstd_post))
    return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t xa = dt_bytes(n.x_dtype);
  if (!aligned(dx_new, xa) || !aligned(x_new, xa) || !aligned(dx, xa) || !aligned(dy, 2) || !aligned(f, 2) ||
      !aligned(df, 2) || !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = nf4moe_block_norm_workspace_bytes(n.H, T);
  if (!ws || ws_bytes < need) return fail(NF4MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  NormArgs a = norm_args(n, T);
  a.x = x_new, a.f = f, a.rstd_post = const_cast<float *>(rstd_post), a.rstd_pre = const_cast<float *>(rstd_pre);
  a.dx_new = dx_new, a.dy = dy, a.dx = dx, a.df = df, a.dgate = dgate;
  a.dw_post = n.w_post ? dw_post : nullptr, a.dw_pre = n.w_pre ? dw_pre : nullptr;
  a.partial = (float *)ws, a.groups = norm_backward_groups(T, n.H);
  return hip_status(launch_norm_backward(a, s), "norm backward launch");
}

}  // extern "C"
