// C ABI of the dense operators (declared in include/nf4moe.h): host-side validation, workspace
// carving and launches. Every check runs before anything is enqueued; on a non-OK status
// nothing was launched.
#include <math.h>

#include "../../include/nf4moe.h"
#include "check.h"
#include "dense.h"
#include "train.h"

using namespace nf4moe;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxHeadRows = (int64_t)1 << 25;   // 64 threads a row (k_head_entries) are inside a dispatch's 2^32
constexpr int kMaxVocab = 1 << 21;   // 256 rows of P are below 2^31 bytes

nf4moe_status_t check_width(int v, const char *name) {
  if (v < 8 || v % 8 || v > kDenseMaxWidth)
    return fail(NF4MOE_ERR_INVALID_ARG, "%s=%d must be a multiple of 8 in 8..%d", name, v, kDenseMaxWidth);
  return NF4MOE_OK;
}

// Sizes whose grids and offsets stay inside a dispatch: tiles of 256 x 256 of a T x n product, and T x n.
nf4moe_status_t check_size(int64_t T, int64_t n) {
  if (T > 0 && (cdiv(T, 256) * cdiv(n, 256) > 1 << 22 || T > ((int64_t)1 << 38) / n))
    return fail(NF4MOE_ERR_UNSUPPORTED, "T=%lld rows of %lld are too many for one call", (long long)T, (long long)n);
  return NF4MOE_OK;
}

nf4moe_status_t check_ffn(const nf4moe_gated_ffn_t *f, int64_t T) {
  if (!f) return fail(NF4MOE_ERR_INVALID_ARG, "ffn is NULL");
  if (T < 0 || T > kMaxRows) return fail(NF4MOE_ERR_INVALID_ARG, "T=%lld outside 0..2^30", (long long)T);
  nf4moe_status_t st = check_width(f->H, "H");
  if (st == NF4MOE_OK) st = check_width(f->I, "I");
  if (st != NF4MOE_OK) return st;
  if (f->glu != NF4MOE_GLU_SWIGLU && f->glu != NF4MOE_GLU_CLAMPED) return fail(NF4MOE_ERR_INVALID_ARG, "unknown glu %d", f->glu);
  if (f->glu == NF4MOE_GLU_CLAMPED &&
      !(f->glu_alpha > 0.0f && f->glu_alpha < 1e30f && f->glu_limit > 0.0f && f->glu_limit < 1e30f))
    return fail(NF4MOE_ERR_INVALID_ARG, "clamped GLU needs finite alpha > 0 and limit > 0");
  if (f->glu_interleaved != 0 && f->glu_interleaved != 1) return fail(NF4MOE_ERR_INVALID_ARG, "glu_interleaved must be 0 or 1");
  st = check_size(T, 2 * (int64_t)f->I);
  if (st == NF4MOE_OK) st = check_size(T, f->H);
  if (st == NF4MOE_OK) st = check_size(2 * (int64_t)f->I, f->H);
  return st;
}

FfnArgs ffn_args(const nf4moe_gated_ffn_t &f, const uint16_t *x, int64_t T) {
  FfnArgs a = {};
  a.T = T, a.H = f.H, a.I = f.I, a.glu = f.glu, a.inter = f.glu_interleaved;
  a.alpha = f.glu_alpha, a.limit = f.glu_limit, a.x = x, a.w13 = f.w13;
  return a;
}

struct FfnCarve {
  uint16_t *dgu, *x2;
  float *part, *wpart;   // slices of dx and of dw13
  int64_t rows;   // of dgu
  size_t bytes;
};
// One size whatever outputs are asked for: that of each alone, which has the most slices.
FfnCarve carve_ffn(void *ws, const nf4moe_gated_ffn_t &f, int64_t T) {
  FfnCarve c = {};
  Bump b{(char *)ws};
  const bool few = T <= kTwoParts;
  c.rows = few ? 2 * T : T;
  c.dgu = b.take<uint16_t>((size_t)c.rows * 2 * f.I);
  if (few) c.x2 = b.take<uint16_t>((size_t)c.rows * f.H);
  const int slices = product_slices(c.rows, f.H, 2 * (int64_t)f.I, true, 8);
  if (few || slices > 1) c.part = b.take<float>((size_t)slices * c.rows * f.H);
  const int wslices = product_slices(2 * (int64_t)f.I, f.H, c.rows, true, 12);
  if (wslices > 1) c.wpart = b.take<float>((size_t)wslices * 2 * f.I * f.H);
  c.bytes = b.off;
  return c;
}

nf4moe_status_t check_head(const nf4moe_head_t *h, int64_t T) {
  if (!h) return fail(NF4MOE_ERR_INVALID_ARG, "head is NULL");
  if (T < 0 || T > kMaxRows) return fail(NF4MOE_ERR_INVALID_ARG, "T=%lld outside 0..2^30", (long long)T);
  nf4moe_status_t st = check_width(h->H, "H");
  if (st != NF4MOE_OK) return st;
  if (h->V < 1 || h->V > kMaxVocab) return fail(NF4MOE_ERR_INVALID_ARG, "V=%d outside 1..%d", h->V, kMaxVocab);
  if (T > kMaxHeadRows) return fail(NF4MOE_ERR_UNSUPPORTED, "T=%lld rows are too many for one call (2^25)", (long long)T);
  st = check_size(T, h->V);
  if (st == NF4MOE_OK) st = check_size(T, h->H);
  if (st == NF4MOE_OK) st = check_size(h->V, h->H);
  return st;
}
nf4moe_status_t check_teacher(int32_t k, float tau) {
  if (k < 1 || k > kMaxTeacher) return fail(NF4MOE_ERR_INVALID_ARG, "k=%d outside 1..%d", k, kMaxTeacher);
  if (!(tau >= 1e-3f && tau <= 1e3f)) return fail(NF4MOE_ERR_INVALID_ARG, "the temperature must lie in 0.001..1000");
  return NF4MOE_OK;
}

struct HeadCarve {
  float2 *stats;
  float *picked;
  uint32_t *list;
  int32_t *offsets;
  uint16_t *P, *x2;
  uint64_t *live;
  float *unit;
  float *part, *wpart;   // slices of dx and of a piece of dw
  int64_t piece, rows;   // rows of P
  size_t bytes;
};
// k: teacher entries a row (0: labels). One size whatever outputs are asked for.
HeadCarve carve_head(void *ws, const nf4moe_head_t &h, int64_t T, int k, bool backward) {
  HeadCarve c = {};
  Bump b{(char *)ws};
  if (k) {
    c.list = b.take<uint32_t>((size_t)cdiv(T, 16) * 16 * k);
    c.offsets = b.take<int32_t>((size_t)cdiv(T, 16) * (cdiv(h.V, kHeadChunk) + 1));
  }
  if (!backward) {
    c.stats = b.take<float2>((size_t)head_stat_chunks(T, h.V, h.H) * T);
    c.picked = b.take<float>(T);
  } else {
    const bool few = T <= kTwoParts;
    c.rows = few ? 2 * T : T;
    c.piece = head_piece(c.rows, h.V);
    c.P = b.take<uint16_t>((size_t)c.rows * c.piece);
    if (few) c.x2 = b.take<uint16_t>((size_t)c.rows * h.H);
    else c.live = b.take<uint64_t>((size_t)cdiv(T, 64)), c.unit = b.take<float>(1);
    const int slices = product_slices(c.rows, h.H, c.piece < h.V ? c.piece : h.V, true, 8);
    if (few || slices > 1 || c.piece < h.V) c.part = b.take<float>((size_t)slices * c.rows * h.H);
    const int64_t most = c.piece < h.V ? c.piece : h.V;
    const int wslices = product_slices(most, h.H, c.rows, true, 12);
    if (wslices > 1) c.wpart = b.take<float>((size_t)wslices * most * h.H);
  }
  c.bytes = b.off;
  return c;
}

nf4moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return fail(NF4MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(NF4MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return NF4MOE_OK;
}

HeadArgs head_args(const nf4moe_head_t &h, const uint16_t *x, int64_t T, const int32_t *ids) {
  HeadArgs a = {};
  a.T = T, a.V = h.V, a.H = h.H, a.tau = 1.0f, a.x = x, a.w = h.w, a.ids = ids;
  return a;
}

// The gradients of either loss, a piece of the vocabulary after the other.
nf4moe_status_t head_backward(HeadArgs a, const HeadCarve &c, uint16_t *dx, uint16_t *dw, hipStream_t s) {
  const bool few = a.T <= kTwoParts;
  const int slices = product_slices(c.rows, a.H, c.piece < a.V ? c.piece : a.V, !dw, 8);
  const bool parts = few || slices > 1 || c.piece < a.V;
  const int wslices = product_slices(c.piece < a.V ? c.piece : a.V, a.H, c.rows, !dx, 12);
  a.P = c.P, a.live = dw ? c.live : nullptr, a.x2 = dw ? c.x2 : nullptr, a.list = c.list, a.offsets = c.offsets, a.unit = c.unit;
  hipError_t e = launch_head_prepare(a, s);
  for (int64_t v0 = 0; v0 < a.V && e == hipSuccess; v0 += c.piece) {
    a.v0 = v0, a.vn = a.V - v0 < c.piece ? a.V - v0 : c.piece, a.vp = c.piece;
    e = launch_head_piece(a, s);
    if (e != hipSuccess) break;
    ProductArgs px = {}, pw = {};
    px.x = a.P, px.ldx = c.piece, px.y = a.w + v0 * a.H, px.ldy = a.H, px.M = c.rows, px.N = a.H, px.K = a.vn;
    px.out = parts ? nullptr : dx, px.part = c.part, px.add = v0 > 0, px.slices = slices;
    pw.x = a.P, pw.ldx = c.piece, pw.y = few ? c.x2 : a.x, pw.ldy = a.H, pw.M = a.vn, pw.N = a.H, pw.K = c.rows;
    pw.out = wslices > 1 ? nullptr : dw + v0 * a.H, pw.part = c.wpart, pw.slices = wslices, pw.live = c.live;
    e = launch_products(dx ? &px : nullptr, dw ? &pw : nullptr, c.unit, s);
    if (e == hipSuccess && dw && wslices > 1) e = launch_join(c.wpart, wslices, a.vn * a.H, c.unit, dw + v0 * a.H, s);
  }
  // (few rows: a slice's second half are the second parts' rows, as one slice more)
  if (e == hipSuccess && dx && parts) e = launch_join(c.part, few ? 2 * slices : slices, a.T * a.H, c.unit, dx, s);
  return hip_status(e, "head backward launch");
}

// What both losses' gradients check and do, `a` with the loss's own arguments.
nf4moe_status_t run_head_backward(const nf4moe_head_t &h, HeadArgs a, const float *dloss, const float *lse, uint16_t *dx,
                                  uint16_t *dw, void *ws, size_t ws_bytes, hipStream_t s) {
  if (!dx && !dw) return fail(NF4MOE_ERR_INVALID_ARG, "neither dx nor dw: nothing to do");
  if (!aligned(dx, 16) || !aligned(dw, 16)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const int64_t T = a.T;
  if (T == 0) return dw ? hip_status(launch_fill_f32_zero((float *)dw, (int64_t)h.V * h.H / 2, s), "fill") : NF4MOE_OK;
  if (!dloss || !a.x || !h.w || !a.ids || !lse) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(a.x, 16) || !aligned(h.w, 16) || !aligned(a.ids, 4) || !aligned(dloss, 4) || !aligned(lse, 4) ||
      !aligned(a.q, 4) || !aligned(a.logits, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const HeadCarve c = carve_head(ws, h, T, a.k, true);
  nf4moe_status_t st = check_ws(ws, ws_bytes, c.bytes);
  if (st != NF4MOE_OK) return st;
  const uint64_t xb = 2 * (uint64_t)T * h.H, wb = 2 * (uint64_t)h.V * h.H, eb = 4 * (uint64_t)T * (a.k ? a.k : 1);
  st = check_overlap({{"dx", dx, xb}, {"dw", dw, wb}, {"workspace", ws, c.bytes}},
                     {{"x", a.x, xb}, {"w", h.w, wb}, {"ids", a.ids, eb}, {"dloss", dloss, 4 * (uint64_t)T},
                      {"lse", lse, 4 * (uint64_t)T}, {"q", a.q, eb}, {"logits", a.logits, eb}});
  if (st != NF4MOE_OK) return st;
  a.dloss = dloss, a.lse = const_cast<float *>(lse);
  return head_backward(a, c, dx, dw, s);
}

nf4moe_status_t check_layer_norm(const nf4moe_layer_norm_t *n, int64_t T) {
  if (!n) return fail(NF4MOE_ERR_INVALID_ARG, "norm is NULL");
  if (T < 0 || T > 0x7fffffff) return fail(NF4MOE_ERR_INVALID_ARG, "T=%lld outside 0..2^31-1", (long long)T);
  if (n->H < 1 || n->H > kLayerNormMaxH) return fail(NF4MOE_ERR_INVALID_ARG, "H=%d outside 1..%d", n->H, kLayerNormMaxH);
  if (!dt_ok(n->x_dtype) || !dt_ok(n->y_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype");
  if (!(n->eps >= 0.0f && n->eps < 1e30f)) return fail(NF4MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!aligned(n->w, 4) || !aligned(n->b, 4)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  return NF4MOE_OK;
}

}  // namespace

extern "C" {

nf4moe_status_t nf4moe_gated_ffn_forward(const nf4moe_gated_ffn_t *ffn, const uint16_t *x, int64_t T, uint16_t *h,
                                         void *stream) {
  nf4moe_status_t st = check_ffn(ffn, T);
  if (st != NF4MOE_OK || T == 0) return st;
  if (!x || !h || !ffn->w13) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, 16) || !aligned(h, 16) || !aligned(ffn->w13, 16)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  st = check_overlap({{"h", h, 2 * (uint64_t)T * ffn->I}},
                     {{"x", x, 2 * (uint64_t)T * ffn->H}, {"w13", ffn->w13, 4 * (uint64_t)ffn->I * ffn->H}});
  if (st != NF4MOE_OK) return st;
  FfnArgs a = ffn_args(*ffn, x, T);
  a.h = h;
  return hip_status(launch_ffn_forward(a, (hipStream_t)stream), "gated feed-forward launch");
}

size_t nf4moe_gated_ffn_workspace_bytes(const nf4moe_gated_ffn_t *ffn, int64_t T) {
  if (T < 1 || check_ffn(ffn, T) != NF4MOE_OK) return 0;
  return carve_ffn(nullptr, *ffn, T).bytes;
}

nf4moe_status_t nf4moe_gated_ffn_backward(const nf4moe_gated_ffn_t *ffn, const uint16_t *dh, const uint16_t *x, int64_t T,
                                          uint16_t *dx, uint16_t *dw13, uint16_t *h, void *ws, size_t ws_bytes,
                                          void *stream) {
  nf4moe_status_t st = check_ffn(ffn, T);
  if (st != NF4MOE_OK) return st;
  if (!dx && !dw13 && T > 0) return fail(NF4MOE_ERR_INVALID_ARG, "neither dx nor dw13: nothing to do");
  if (!aligned(dx, 16) || !aligned(dw13, 16) || !aligned(h, 16)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const nf4moe_gated_ffn_t &f = *ffn;
  hipStream_t s = (hipStream_t)stream;
  const int64_t cells = (int64_t)f.I * f.H;
  if (T == 0) return dw13 ? hip_status(launch_fill_f32_zero((float *)dw13, cells, s), "fill") : NF4MOE_OK;
  if (!dh || !x || !f.w13) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(dh, 16) || !aligned(x, 16) || !aligned(f.w13, 16)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const FfnCarve c = carve_ffn(ws, f, T);
  st = check_ws(ws, ws_bytes, c.bytes);
  if (st != NF4MOE_OK) return st;
  const uint64_t xb = 2 * (uint64_t)T * f.H, hb = 2 * (uint64_t)T * f.I, wb = 4 * (uint64_t)cells;
  st = check_overlap({{"dx", dx, xb}, {"dw13", dw13, wb}, {"h", h, hb}, {"workspace", ws, c.bytes}},
                     {{"dh", dh, hb}, {"x", x, xb}, {"w13", f.w13, wb}});
  if (st != NF4MOE_OK) return st;
  FfnArgs a = ffn_args(f, x, T);
  a.dh = dh, a.dgu = c.dgu, a.h = h, a.x2 = dw13 ? c.x2 : nullptr;
  hipError_t e = launch_ffn_dgu(a, s);
  const bool few = T <= kTwoParts;
  const int slices = product_slices(c.rows, f.H, 2 * (int64_t)f.I, !dw13, 8);
  const bool parts = few || slices > 1;
  const int wslices = product_slices(2 * (int64_t)f.I, f.H, c.rows, !dx, 12);
  ProductArgs px = {}, pw = {};
  px.x = c.dgu, px.ldx = 2 * (int64_t)f.I, px.y = f.w13, px.ldy = f.H, px.M = c.rows, px.N = f.H, px.K = 2 * (int64_t)f.I;
  px.out = parts ? nullptr : dx, px.part = c.part, px.slices = slices;
  pw.x = c.dgu, pw.ldx = 2 * (int64_t)f.I, pw.y = few ? c.x2 : x, pw.ldy = f.H, pw.M = 2 * (int64_t)f.I, pw.N = f.H, pw.K = c.rows;
  pw.out = wslices > 1 ? nullptr : dw13, pw.part = c.wpart, pw.slices = wslices;
  if (e == hipSuccess) e = launch_products(dx ? &px : nullptr, dw13 ? &pw : nullptr, nullptr, s);
  // (few rows: a slice's second half are the second parts' rows, as one slice more)
  if (e == hipSuccess && dx && parts) e = launch_join(c.part, few ? 2 * slices : slices, T * f.H, nullptr, dx, s);
  if (e == hipSuccess && dw13 && wslices > 1) e = launch_join(c.wpart, wslices, 2 * cells, nullptr, dw13, s);
  return hip_status(e, "gated feed-forward backward launch");
}

size_t nf4moe_vocab_workspace_bytes(const nf4moe_head_t *head, int64_t T, int32_t k, int32_t backward) {
  if (T < 1 || k < 0 || k > kMaxTeacher || check_head(head, T) != NF4MOE_OK) return 0;
  return carve_head(nullptr, *head, T, k, backward != 0).bytes;
}

nf4moe_status_t nf4moe_vocab_ce_forward(const nf4moe_head_t *head, const uint16_t *x, int64_t T, const int32_t *labels,
                                        float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_head(head, T);
  if (st != NF4MOE_OK || T == 0) return st;
  if (!x || !head->w || !labels || !loss || !lse) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, 16) || !aligned(head->w, 16) || !aligned(labels, 4) || !aligned(loss, 4) || !aligned(lse, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const HeadCarve c = carve_head(ws, *head, T, 0, false);
  st = check_ws(ws, ws_bytes, c.bytes);
  if (st != NF4MOE_OK) return st;
  const uint64_t rows = 4 * (uint64_t)T;
  st = check_overlap({{"loss", loss, rows}, {"lse", lse, rows}, {"workspace", ws, c.bytes}},
                     {{"x", x, 2 * (uint64_t)T * head->H}, {"w", head->w, 2 * (uint64_t)head->V * head->H}, {"labels", labels, rows}});
  if (st != NF4MOE_OK) return st;
  HeadArgs a = head_args(*head, x, T, labels);
  a.loss = loss, a.lse = lse, a.stats = c.stats, a.picked = c.picked;
  return hip_status(launch_head_forward(a, (hipStream_t)stream), "head launch");
}

nf4moe_status_t nf4moe_vocab_ce_backward(const nf4moe_head_t *head, const float *dloss, const uint16_t *x, int64_t T,
                                         const int32_t *labels, const float *lse, uint16_t *dx, uint16_t *dw, void *ws,
                                         size_t ws_bytes, void *stream) {
  const nf4moe_status_t st = check_head(head, T);
  if (st != NF4MOE_OK) return st;
  return run_head_backward(*head, head_args(*head, x, T, labels), dloss, lse, dx, dw, ws, ws_bytes, (hipStream_t)stream);
}

nf4moe_status_t nf4moe_vocab_distill_forward(const nf4moe_head_t *head, const uint16_t *x, int64_t T, const int32_t *ids,
                                             const void *teacher, nf4moe_dtype_t teacher_dtype, int32_t k,
                                             float temperature, float *loss, float *lse, float *q, float *logits, void *ws,
                                             size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_head(head, T);
  if (st == NF4MOE_OK) st = check_teacher(k, temperature);
  if (st != NF4MOE_OK) return st;
  if (!dt_ok(teacher_dtype)) return fail(NF4MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)teacher_dtype);
  if (T == 0) return NF4MOE_OK;
  if (!x || !head->w || !ids || !teacher || !loss || !lse || !q || !logits) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, 16) || !aligned(head->w, 16) || !aligned(ids, 4) || !aligned(teacher, dt_bytes(teacher_dtype)) ||
      !aligned(loss, 4) || !aligned(lse, 4) || !aligned(q, 4) || !aligned(logits, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const HeadCarve c = carve_head(ws, *head, T, k, false);
  st = check_ws(ws, ws_bytes, c.bytes);
  if (st != NF4MOE_OK) return st;
  const uint64_t rows = 4 * (uint64_t)T, n = (uint64_t)T * k;
  st = check_overlap({{"loss", loss, rows}, {"lse", lse, rows}, {"q", q, 4 * n}, {"logits", logits, 4 * n}, {"workspace", ws, c.bytes}},
                     {{"x", x, 2 * (uint64_t)T * head->H}, {"w", head->w, 2 * (uint64_t)head->V * head->H}, {"ids", ids, 4 * n},
                      {"teacher", teacher, n * dt_bytes(teacher_dtype)}});
  if (st != NF4MOE_OK) return st;
  HeadArgs a = head_args(*head, x, T, ids);
  a.k = k, a.tau = temperature, a.teacher = teacher, a.teacher_bf16 = teacher_dtype == NF4MOE_DT_BF16;
  a.loss = loss, a.lse = lse, a.q = q, a.logits = logits, a.stats = c.stats, a.list = c.list, a.offsets = c.offsets;
  return hip_status(launch_head_forward(a, (hipStream_t)stream), "head launch");
}

nf4moe_status_t nf4moe_vocab_distill_backward(const nf4moe_head_t *head, const float *dloss, const uint16_t *x, int64_t T,
                                              const int32_t *ids, const float *q, const float *logits, const float *lse,
                                              int32_t k, float temperature, uint16_t *dx, uint16_t *dw, void *ws,
                                              size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_head(head, T);
  if (st == NF4MOE_OK) st = check_teacher(k, temperature);
  if (st != NF4MOE_OK) return st;
  if (T > 0 && (!q || !logits)) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  HeadArgs a = head_args(*head, x, T, ids);
  a.k = k, a.tau = temperature, a.q = const_cast<float *>(q), a.logits = const_cast<float *>(logits);
  return run_head_backward(*head, a, dloss, lse, dx, dw, ws, ws_bytes, (hipStream_t)stream);
}

nf4moe_status_t nf4moe_layer_norm_forward(const nf4moe_layer_norm_t *norm, const void *x, int64_t T, void *y, float *mean,
                                          float *rstd, void *stream) {
  nf4moe_status_t st = check_layer_norm(norm, T);
  if (st != NF4MOE_OK || T == 0) return st;
  const nf4moe_layer_norm_t &n = *norm;
  if (!x || !y || !mean || !rstd) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t xe = dt_bytes(n.x_dtype), ye = dt_bytes(n.y_dtype);
  if (!aligned(x, xe) || !aligned(y, ye) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const uint64_t rows = (uint64_t)T, cells = rows * n.H, wb = 4 * (uint64_t)n.H;
  st = check_overlap({{"y", y, cells * ye}, {"mean", mean, 4 * rows}, {"rstd", rstd, 4 * rows}},
                     {{"x", x, cells * xe}, {"w", n.w, wb}, {"b", n.b, wb}});
  if (st != NF4MOE_OK) return st;
  LayerNormArgs a = {};
  a.T = T, a.H = n.H, a.x_bf16 = n.x_dtype == NF4MOE_DT_BF16, a.y_bf16 = n.y_dtype == NF4MOE_DT_BF16;
  a.x = x, a.w = n.w, a.b = n.b, a.eps = n.eps, a.y = y, a.mean = mean, a.rstd = rstd;
  return hip_status(launch_layer_norm_forward(a, (hipStream_t)stream), "layer norm launch");
}

size_t nf4moe_layer_norm_workspace_bytes(int32_t H, int64_t T) {
  if (H < 1 || H > kLayerNormMaxH || T < 1 || T > 0x7fffffff) return 0;
  return align_up((size_t)layer_norm_groups(T, H) * 2 * H * sizeof(float));
}

nf4moe_status_t nf4moe_layer_norm_backward(const nf4moe_layer_norm_t *norm, const void *dy, const void *x, const float *mean,
                                           const float *rstd, int64_t T, const void *dx_base, void *dx, float *dw, float *db,
                                           void *ws, size_t ws_bytes, void *stream) {
  nf4moe_status_t st = check_layer_norm(norm, T);
  if (st != NF4MOE_OK) return st;
  const nf4moe_layer_norm_t &n = *norm;
  if (!dx && !dw && !db && T > 0) return fail(NF4MOE_ERR_INVALID_ARG, "neither dx, dw nor db: nothing to do");
  if (!aligned(dw, 4) || !aligned(db, 4)) return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) {  // the sums over no rows
    hipError_t e = hipSuccess;
    if (dw) e = launch_fill_i32((int32_t *)dw, n.H, 0, s);
    if (e == hipSuccess && db) e = launch_fill_i32((int32_t *)db, n.H, 0, s);
    return hip_status(e, "fill");
  }
  if (!dy || !x || !mean || !rstd) return fail(NF4MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t xe = dt_bytes(n.x_dtype), ye = dt_bytes(n.y_dtype);
  if (!aligned(dy, ye) || !aligned(x, xe) || !aligned(dx_base, xe) || !aligned(dx, xe) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(NF4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = nf4moe_layer_norm_workspace_bytes(n.H, T);
  st = check_ws(ws, ws_bytes, need);
  if (st != NF4MOE_OK) return st;
  const uint64_t rows = (uint64_t)T, cells = rows * n.H, wb = 4 * (uint64_t)n.H;
  st = check_overlap({{"dx", dx, cells * xe}, {"dw", dw, wb}, {"db", db, wb}, {"workspace", ws, need}},
                     {{"dy", dy, cells * ye}, {"x", x, cells * xe}, but({"dx_base", dx_base, cells * xe}, dx),
                      {"mean", mean, 4 * rows}, {"rstd", rstd, 4 * rows}, {"w", n.w, wb}});
  if (st != NF4MOE_OK) return st;
  LayerNormArgs a = {};
  a.T = T, a.H = n.H, a.x_bf16 = n.x_dtype == NF4MOE_DT_BF16, a.y_bf16 = n.y_dtype == NF4MOE_DT_BF16;
  a.x = x, a.w = n.w, a.eps = n.eps, a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
  a.dy = dy, a.dx_base = dx_base, a.dx = dx, a.dw = dw, a.db = db;
  a.partial = (float *)ws, a.groups = layer_norm_groups(T, n.H);
  return hip_status(launch_layer_norm_backward(a, s), "layer norm backward launch");
}

}  // extern "C"
