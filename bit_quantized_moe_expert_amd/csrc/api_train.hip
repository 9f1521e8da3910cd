// C ABI of the fine-tuning operators (declared in include/nf4moe.h): host-side
// validation, workspace carving and launches. Every check runs before anything
// is enqueued; on a non-OK status nothing was launched.
#include <math.h>

#include <initializer_list>

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

// An array that a call writes or reads (absent: no address or no bytes).
struct Span {
  const char *name;
  const void *p;
  uint64_t n;
};
bool overlap(const Span &a, const Span &b) {
  const uint64_t p = (uint64_t)a.p, q = (uint64_t)b.p;
  return p && q && a.n && b.n && p < q + b.n && q < p + a.n;
}

// No output shares a byte with an input or with another output. An input that an output
// may be is left out of `ins` by the caller where it is that very array (see but()).
nf4moe_status_t check_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *o = outs.begin(); o != outs.end(); ++o) {
    for (const Span *q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return fail(NF4MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
    for (const Span &q : ins)
      if (overlap(*o, q)) return fail(NF4MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q.name);
  }
  return NF4MOE_OK;
}
Span but(Span in, const void *out) { return {in.name, in.p == out ? nullptr : in.p, in.n}; }

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
  // the kernels count the 2 I columns of a row in 32 bits, up to 2 I - 8 and 8 values from there
  if (I > 1 << 30) return fail(NF4MOE_ERR_UNSUPPORTED, "I=%d past 2^30", I);
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

// Elements of a gate, and of its gradient.
uint64_t gate_count(const nf4moe_block_norm_t &n, int64_t T) {
  const uint64_t count[4] = {0, (uint64_t)n.H, (uint64_t)T, (uint64_t)T * n.H};
  return count[n.gate_kind];
}

NormArgs norm_args(const nf4moe_block_norm_t &n, int64_t T) {
  NormArgs a = {};
  a.T = T, a.H = n.H, a.x_bf16 = n.x_dtype == NF4MOE_DT_BF16;
  a.w_post = n.w_post, a.w_pre = n.w_pre;
  a.gate = n.gate, a.gate_kind = n.gate_kind, a.gate_bf16 = n.gate_dtype == NF4MOE_DT_BF16, a.gate_fn = n.gate_fn;
  a.alpha = n.alpha, a.eps = n.eps;
  return a;
}

nf4moe_status_t check_adapters(const nf4moe_adapters_t *a, int64_t R) {
  if (!a) return fail(NF4MOE_ERR_INVALID_ARG, "adapters is NULL");
  if (a->L < 1 || a->L > kMaxAdapters) return fail(NF4MOE_ERR_INVALID_ARG, "L=%d outside 1..%d", a->L, kMaxAdapters);
  if (a->rank < 8 || a->rank > kMaxRank || a->rank % 8)
    return fail(NF4MOE_ERR_INVALID_ARG, "rank=%d must be a multiple of 8 in 8..%d", a->rank, kMaxRank);
  if (a->K < 8 || a->K % 8 || a->K > (1 << 20) || a->N < 8 || a->N % 8 || a->N > (1 << 20))
    return fail(NF4MOE_ERR_INVALID_ARG, "K=%d and N=%d must be multiples of 8 in 8..2^20", a->K, a->N);
  if (R < 0 || R > (1 << 30)) return fail(NF4MOE_ERR_INVALID_ARG, "R=%lld outside 0..2^30", (long long)R);
  if (R > 0 && (!a->A || !a->B)) return fail(NF4MOE_ERR_INVALID_ARG, "adapter weight pointer is NULL");
  if (!aligned(a->A, 2) || !aligned(a->B, 2) || !aligned(a->scale, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  return NF4MOE_OK;
}

// Bump allocator over the caller's workspace (sizes alone with a null base).
struct Bump {
  char *base;
  size_t off = 0;
  template <class T>
  T *take(size_t count) {
    T *p = base ? (T *)(base + off) : nullptr;
    off = align_up(off + count * sizeof(T));
    return p;
  }
};

struct AdapterCarve {
  void *plan;
  float *slices;                // partial low-rank products
  uint16_t *parts;              // the low-rank product for the second one
  float *u;                     // backward: [R, rank]
  uint16_t *At, *Bt;            // [L, K, rank], [L, rank, N]
  float *partial_a, *partial_b;
  size_t bytes;
};

// The calls' scratch: with `plan` given by the caller its part is left out; the
// rest has one size whatever outputs are asked for.
AdapterCarve carve_adapter(void *ws, const nf4moe_adapters_t &a, int R, bool backward) {
  AdapterCarve c = {};
  Bump b{(char *)ws};
  AdapterPlan lay;
  c.plan = b.take<char>(adapter_plan_layout(R, a.L, nullptr, &lay));
  c.slices = b.take<float>((size_t)adapter_slices(R, backward ? a.N : a.K, a.rank) * R * a.rank);
  c.parts = b.take<uint16_t>(adapter_parts_elems(lay.max_tiles, a.rank));
  if (backward) {
    c.u = b.take<float>((size_t)R * a.rank);
    c.At = b.take<uint16_t>((size_t)a.L * a.K * a.rank);
    c.Bt = b.take<uint16_t>((size_t)a.L * a.N * a.rank);
    c.partial_a = b.take<float>((size_t)lay.max_slots * a.rank * a.K);
    c.partial_b = b.take<float>((size_t)lay.max_slots * a.rank * a.N);
  }
  c.bytes = b.off;
  return c;
}

}  // namespace

extern "C" {

nf4moe_status_t nf4moe_ckpt8_quantize(nf4moe_ckpt8_t fmt, const void *x, nf4moe_dtype_t x_dtype, int64_t rows, int64_t K,
                                      uint8_t *codes, uint8_t *scale, void *stream) {
  const nf4moe_status_t st = check_ckpt8(fmt, x, x_dtype, rows, K, codes, scale);
  if (st != NF4MOE_OK || rows == 0) return st;
  const uint64_t n = (uint64_t)rows * K;
  const nf4moe_status_t apart = check_overlap({{"codes", codes, n}, {"scale", scale, n / 32}}, {{"x", x, n * dt_bytes(x_dtype)}});
  if (apart != NF4MOE_OK) return apart;
  return hip_status(launch_ckpt8_quantize(fmt, x, x_dtype == NF4MOE_DT_BF16, rows * K, codes, scale, (hipStream_t)stream),
                    "checkpoint quantize launch");
}

nf4moe_status_t nf4moe_ckpt8_dequantize(nf4moe_ckpt8_t fmt, const uint8_t *codes, const uint8_t *scale, int64_t rows,
                                        int64_t K, void *out, nf4moe_dtype_t out_dtype, void *stream) {
  const nf4moe_status_t st = check_ckpt8(fmt, out, out_dtype, rows, K, codes, scale);
  if (st != NF4MOE_OK || rows == 0) return st;
  const uint64_t n = (uint64_t)rows * K;
  const nf4moe_status_t apart = check_overlap({{"out", out, n * dt_bytes(out_dtype)}}, {{"codes", codes, n}, {"scale", scale, n / 32}});
  if (apart != NF4MOE_OK) return apart;
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
  const uint64_t n = (uint64_t)R * I;
  const nf4moe_status_t apart = check_overlap({{"h", h, 2 * n}, {"codes", codes, 2 * n}, {"scale", scale, n / 16}},
                                              {{"gu", gu, 2 * n * dt_bytes(gu_dtype)}});
  if (apart != NF4MOE_OK) return apart;
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
  const uint64_t n = (uint64_t)R * I;
  const nf4moe_status_t apart = check_overlap(
      {{"dgu", dgu, 4 * n}, {"h", h, 2 * n}, {"drow_w", drow_w, 4 * (uint64_t)R}},
      {{"dh", dh, n * dt_bytes(dh_dtype)}, {"gu", gu, 2 * n * (held ? 1 : gu_src == NF4MOE_SRC_F32 ? 4 : 2)},
       {"gu_scale", held ? gu_scale : nullptr, n / 16}, {"row_w", row_w, 4 * (uint64_t)R}});
  if (apart != NF4MOE_OK) return apart;
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
  const uint64_t rows = (uint64_t)T, cells = rows * n.H, xb = cells * dt_bytes(n.x_dtype), wb = 4 * (uint64_t)n.H;
  const nf4moe_status_t apart = check_overlap(
      {{"x_new", f ? x_new : nullptr, xb}, {"y", n.w_pre ? y : nullptr, 2 * cells},
       {"rstd_post", n.w_post ? rstd_post : nullptr, 4 * rows}, {"rstd_pre", n.w_pre ? rstd_pre : nullptr, 4 * rows}},
      {but({"x", x, xb}, f ? x_new : nullptr), {"f", f, 2 * cells}, {"w_post", n.w_post, wb}, {"w_pre", n.w_pre, wb},
       {"gate", n.gate, gate_count(n, T) * dt_bytes(n.gate_dtype)}});
  if (apart != NF4MOE_OK) return apart;
  NormArgs a = norm_args(n, T);
  a.x = x, a.f = f, a.x_new = x_new, a.y = y, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
  return hip_status(launch_norm_forward(a, (hipStream_t)stream), "norm launch");
}

size_t nf4moe_block_norm_workspace_bytes(int32_t H, int64_t T) {
  if (H < 1 || H > kNormMaxH || T < 1 || T > 0x7fffffff) return 0;
  return align_up((size_t)norm_backward_groups(T, H) * 2 * H * sizeof(float));
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
  const uint64_t rows = (uint64_t)T, cells = rows * n.H, xb = cells * xa, wb = 4 * (uint64_t)n.H;
  const nf4moe_status_t apart = check_overlap(
      {{"dx", dx, xb}, {"df", f ? df : nullptr, 2 * cells}, {"dgate", n.gate ? dgate : nullptr, 4 * gate_count(n, T)},
       {"dw_post", n.w_post ? dw_post : nullptr, wb}, {"dw_pre", n.w_pre ? dw_pre : nullptr, wb}, {"workspace", ws, need}},
      {{"dx_new", dx_new, xb}, {"dy", n.w_pre ? dy : nullptr, 2 * cells}, {"x_new", n.w_pre ? x_new : nullptr, xb},
       {"f", f, 2 * cells}, {"rstd_post", n.w_post ? rstd_post : nullptr, 4 * rows},
       {"rstd_pre", n.w_pre ? rstd_pre : nullptr, 4 * rows}, {"w_post", n.w_post, wb}, {"w_pre", n.w_pre, wb},
       {"gate", n.gate, gate_count(n, T) * dt_bytes(n.gate_dtype)}});
  if (apart != NF4MOE_OK) return apart;
  NormArgs a = norm_args(n, T);
  a.x = x_new, a.f = f, a.rstd_post = const_cast<float *>(rstd_post), a.rstd_pre = const_cast<float *>(rstd_pre);
  a.dx_new = dx_new, a.dy = dy, a.dx = dx, a.df = df, a.dgate = dgate;
  a.dw_post = n.w_post ? dw_post : nullptr, a.dw_pre = n.w_pre ? dw_pre : nullptr;
  a.partial = (float *)ws, a.groups = norm_backward_groups(T, n.H);
  return hip_status(launch_norm_backward(a, s), "norm backward launch");
}

size_t nf4moe_adapter_plan_bytes(int32_t R, int32_t L) {
  if (R < 1 || R > (1 << 30) || L < 1 || L > kMaxAdapters) return 0;
  return adapter_plan_layout(R, L, nullptr, nullptr);
}

nf4moe_status_t nf4moe_adapter_plan(const int32_t *ids, int32_t R, int32_t L, void *plan, size_t plan_bytes, void *stream) {
  if (L < 1 || L > kMaxAdapters) return fail(NF4MOE_ERR_INVALID_ARG, "L=%d outside 1..%d", L, kMaxAdapters);
  if (R < 0 || R > (1 << 30)) return fail(NF4MOE_ERR_INVALID_ARG, "R=%d outside 0..2^30", R);
  if (R == 0) return NF4MOE_OK;
  if (!ids) return fail(NF4MOE_ERR_INVALID_ARG, "ids is NULL");
  if (!aligned(ids, 4)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = nf4moe_adapter_plan_bytes(R, L);
  if (!plan || plan_bytes < need) return fail(NF4MOE_ERR_WORKSPACE, "plan %zu bytes < %zu required", plan_bytes, need);
  if (!aligned(plan, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "plan must be 256-byte aligned");
  const nf4moe_status_t apart = check_overlap({{"plan", plan, need}}, {{"ids", ids, 4 * (uint64_t)R}});
  if (apart != NF4MOE_OK) return apart;
  AdapterPlan p;
  adapter_plan_layout(R, L, plan, &p);
  return hip_status(launch_adapter_prepare({p, ids, R, L, 0, 0, 0, nullptr, nullptr, nullptr, nullptr}, (hipStream_t)stream), "adapter plan launch");
}

size_t nf4moe_adapter_workspace_bytes(const nf4moe_adapters_t *ad, int32_t R, int32_t backward) {
  if (!ad || R < 1 || R > (1 << 30) || ad->L < 1 || ad->L > kMaxAdapters || ad->rank < 8 || ad->rank > kMaxRank ||
      ad->K < 8 || ad->N < 8)
    return 0;
  if (!backward && adapter_rows_supported(R, ad->K, ad->N, ad->rank)) return 0;
  return carve_adapter(nullptr, *ad, R, backward != 0).bytes;
}

// Rows, gather, ids and plan, as both directions take them; `cols` is the width that
// is written, dA's and dB's included. Grids reach a workgroup of 256 threads per 64
// rows, or per adapter, and 128 columns; a dispatch holds less than 2^32 threads.
static nf4moe_status_t check_adapter_rows(int32_t R, int32_t x_rows, const int32_t *x_row_of, const int32_t *ids,
                                          const void *plan, size_t plan_bytes, int32_t L, int64_t cols, bool sums) {
  const int64_t tiles = cdiv(R, kAdTile) + (R < L + 1 && !sums ? R : L + 1), per = cdiv(cols, 128) + 1;
  if (tiles * (per < 8 ? 8 : per) >= 1 << 24)
    return fail(NF4MOE_ERR_UNSUPPORTED, "R=%d rows of %lld columns are too many for one call", R, (long long)cols);
  if (x_rows < 1 || (!x_row_of && x_rows < R))
    return fail(NF4MOE_ERR_INVALID_ARG, "x_rows=%d too small for R=%d%s", x_rows, R, x_row_of ? "" : " without a gather");
  if (!ids) return fail(NF4MOE_ERR_INVALID_ARG, "ids is NULL");
  if (!aligned(ids, 4) || !aligned(x_row_of, 4)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (plan) {
    if (plan_bytes < nf4moe_adapter_plan_bytes(R, L))
      return fail(NF4MOE_ERR_WORKSPACE, "plan %zu bytes < %zu required", plan_bytes, nf4moe_adapter_plan_bytes(R, L));
    if (!aligned(plan, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "plan must be 256-byte aligned");
  }
  return NF4MOE_OK;
}

nf4moe_status_t nf4moe_adapter_forward(const nf4moe_adapters_t *ad, const uint16_t *x, int32_t x_rows,
                                       const int32_t *x_row_of, const int32_t *ids, const void *plan, size_t plan_bytes,
                                       int32_t R, const void *base, void *out, nf4moe_dtype_t dtype, float *t, void *ws,
                                       size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_adapters(ad, R);
  if (st != NF4MOE_OK) return st;
  if (!dt_ok(dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (R == 0) return NF4MOE_OK;
  if ((st = check_adapter_rows(R, x_rows, x_row_of, ids, plan, plan_bytes, ad->L, ad->N, false)) != NF4MOE_OK) return st;
  if (!x || !out) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, 2) || !aligned(base, dt_bytes(dtype)) || !aligned(out, dt_bytes(dtype)) || !aligned(t, 16))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  hipStream_t s = (hipStream_t)stream;
  const bool bf = dtype == NF4MOE_DT_BF16;
  const bool one_launch = adapter_rows_supported(R, ad->K, ad->N, ad->rank);
  const size_t need = one_launch ? 0 : carve_adapter(nullptr, *ad, R, false).bytes;
  if (!one_launch) {
    if (!ws || ws_bytes < need) return fail(NF4MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
    if (!aligned(ws, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  const uint64_t rows = (uint64_t)R, ob = rows * ad->N * dt_bytes(dtype), lr = (uint64_t)ad->L * ad->rank * 2;
  st = check_overlap({{"out", out, ob}, {"t", t, 4 * rows * ad->rank}, {"workspace", ws, need}},
                     {{"x", x, (uint64_t)x_rows * ad->K * 2}, {"x_row_of", x_row_of, 4 * rows}, {"ids", ids, 4 * rows},
                      {"plan", plan, nf4moe_adapter_plan_bytes(R, ad->L)}, but({"base", base, ob}, out), {"A", ad->A, lr * ad->K}, {"B", ad->B, lr * ad->N},
                      {"scale", ad->scale, 4 * (uint64_t)ad->L}});
  if (st != NF4MOE_OK) return st;
  if (one_launch) {
    AdapterRowsArgs a = {x, x_row_of, ids, x_rows, R, ad->L, ad->K, ad->N, ad->rank, ad->A, ad->B, ad->scale, base, out, bf, t};
    return hip_status(launch_adapter_rows(a, s), "adapter launch");
  }
  const AdapterCarve c = carve_adapter(ws, *ad, R, false);
  AdapterPlan p;
  adapter_plan_layout(R, ad->L, plan ? const_cast<void *>(plan) : c.plan, &p);
  hipError_t e = plan ? hipSuccess : launch_adapter_prepare({p, ids, R, ad->L, 0, 0, 0, nullptr, nullptr, nullptr, nullptr}, s);
  if (e != hipSuccess) return hip_status(e, "adapter plan launch");
  const LowRankArgs a = {p, R, x, x_row_of, x_rows, ad->A, ad->B, ad->scale, ad->K, ad->N, ad->rank,
                         t, false, base, out, bf, c.slices, c.parts};
  e = launch_adapter_shrink(a, s);
  return hip_status(e != hipSuccess ? e : launch_adapter_expand(a, s), "adapter launch");
}

nf4moe_status_t nf4moe_adapter_backward(const nf4moe_adapters_t *ad, const uint16_t *dy, nf4moe_src_t x_src, const void *x,
                                        const uint8_t *x_scale, int32_t x_rows, const int32_t *x_row_of, const float *t,
                                        const int32_t *ids, const void *plan, size_t plan_bytes, int32_t R,
                                        const void *dx_base, void *dx, nf4moe_dtype_t dx_dtype, float *dA, float *dB,
                                        void *ws, size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_adapters(ad, R);
  if (st != NF4MOE_OK) return st;
  if (!dt_ok(dx_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dx_dtype);
  if (x_src < NF4MOE_SRC_BF16 || x_src > NF4MOE_SRC_MXFP8)
    return fail(NF4MOE_ERR_INVALID_ARG, "x must be bf16 or an 8-bit checkpoint, got source %d", (int)x_src);
  const bool held = x_src >= NF4MOE_SRC_MXINT8;
  if (held && ad->K % 32) return fail(NF4MOE_ERR_INVALID_ARG, "an 8-bit x needs K %% 32 == 0 (K=%d)", ad->K);
  if (!aligned(dA, 16) || !aligned(dB, 16)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (R == 0) {  // sums over no rows
    if (dA) e = launch_fill_f32_zero(dA, (int64_t)ad->L * ad->rank * ad->K, s);
    if (e == hipSuccess && dB) e = launch_fill_f32_zero(dB, (int64_t)ad->L * ad->rank * ad->N, s);
    return hip_status(e, "fill launch");
  }
  st = check_adapter_rows(R, dA ? x_rows : R, x_row_of, ids, plan, plan_bytes, ad->L, (int64_t)ad->K + ad->N, dA || dB);
  if (st != NF4MOE_OK) return st;
  if (!dy || (dA && (!x || (held && !x_scale))) || (dB && !t)) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(dy, 2) || !aligned(x, held ? 1 : 2) || !aligned(t, 16) || !aligned(dx_base, dt_bytes(dx_dtype)) ||
      !aligned(dx, dt_bytes(dx_dtype)))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const AdapterCarve need = carve_adapter(nullptr, *ad, R, true);
  if (!ws || ws_bytes < need.bytes)
    return fail(NF4MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need.bytes);
  if (!aligned(ws, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!dx && !dA && !dB) return NF4MOE_OK;
  const uint64_t rows = (uint64_t)R, xb = rows * ad->K * dt_bytes(dx_dtype), lr = (uint64_t)ad->L * ad->rank * 2;
  const uint64_t held_x = dA ? (uint64_t)x_rows * ad->K : 0;
  st = check_overlap({{"dx", dx, xb}, {"dA", dA, 2 * lr * ad->K}, {"dB", dB, 2 * lr * ad->N}, {"workspace", ws, need.bytes}},
                     {{"dy", dy, 2 * rows * ad->N}, {"x", x, held ? held_x : 2 * held_x},
                      {"x_scale", held ? x_scale : nullptr, held_x / 32}, {"x_row_of", x_row_of, 4 * rows},
                      {"t", dB ? t : nullptr, 4 * rows * ad->rank}, {"ids", ids, 4 * rows}, {"plan", plan, nf4moe_adapter_plan_bytes(R, ad->L)},
                      but({"dx_base", dx ? dx_base : nullptr, xb}, dx), {"A", ad->A, lr * ad->K}, {"B", ad->B, lr * ad->N},
                      {"scale", ad->scale, 4 * (uint64_t)ad->L}});
  if (st != NF4MOE_OK) return st;
  const AdapterCarve c = carve_adapter(ws, *ad, R, true);
  AdapterPlan p;
  adapter_plan_layout(R, ad->L, plan ? const_cast<void *>(plan) : c.plan, &p);
  // u = s B^T dy and dx = dx_base + A^T u: the forward's kernels on B as [L, rank, N]
  // and A as [L, K, rank]
  e = launch_adapter_prepare({p, plan ? nullptr : ids, R, ad->L, ad->K, ad->N, ad->rank, ad->A, ad->B, dx ? c.At : nullptr,
                              dx || dA ? c.Bt : nullptr}, s);
  if (e != hipSuccess) return hip_status(e, "adapter prepare launch");
  const LowRankArgs a = {p, R, dy, nullptr, R, c.Bt, c.At, ad->scale, ad->N, ad->K, ad->rank, dA ? c.u : nullptr, true,
                         dx_base, dx, dx_dtype == NF4MOE_DT_BF16, c.slices, dx ? c.parts : nullptr};
  if (dx || dA) {
    e = launch_adapter_shrink(a, s);
    if (e != hipSuccess) return hip_status(e, "adapter backward launch");
  }
  if (dA || dB) {
    RowGradArgs g = {p, R, ad->L, ad->rank, x_src, {}, {}};
    g.a = {c.u, x, x_scale, x_row_of, x_rows, nullptr, ad->K, false, dA, c.partial_a};
    g.b = {t, dy, nullptr, nullptr, R, ad->scale, ad->N, true, dB, c.partial_b};
    e = launch_adapter_rowgrad(g, s);
    if (e != hipSuccess) return hip_status(e, "adapter weight gradient launch");
  }
  // after dB, which finds dy (up to the last-level cache's size) where u's product left it
  return dx ? hip_status(launch_adapter_expand(a, s), "adapter backward launch") : NF4MOE_OK;
}

}  // extern "C"
