/*
 * nf4moe.h -- C ABI of libnf4moe.so: the routed Mixture-of-Experts expert layer
 * computed directly on 4-bit packed weights, for AMD Instinct MI355X (gfx950).
 *
 * The operation is the one described on the page "How do I run a grouped GEMM
 * directly on NF4 packed MoE expert weights, without dequantizing to bf16
 * first?" (sections "Why it happens", "Smallest correct example", "Supported
 * scope") and in the grouped-nf4-gemm PKG-INFO (intro, "Try it on CPU right
 * now", "The MXFP4 native-byte lane"): one grouped GEMM over an expert-major
 * stack of 4-bit codes, each code decoded through a 16-entry codebook in
 * registers, block-scaled, accumulated in fp32, with no bf16 copy of any expert
 * written to memory. This library also does the routing (router logits, top-k,
 * grouping) and the router-weighted combine, so one call runs a whole layer.
 *
 * Conventions for every entry point
 *  - Pointers marked "device" are HIP device memory owned by the caller. The
 *    library allocates no device memory and keeps no state between calls; the
 *    scratch an operation needs is a caller-provided workspace.
 *  - stream: a hipStream_t (NULL = the null stream). All device work is
 *    enqueued asynchronously on it; no call synchronises the host, so the
 *    forward pass can be captured in a HIP graph.
 *  - Every argument is validated on the host before anything is enqueued; on
 *    an error nothing is enqueued, the status is returned and
 *    nf4moe_last_error() (thread-local) describes it.
 *  - Element offsets are computed in 64 bits everywhere, so expert stacks may
 *    exceed 2 GiB (the pages' "Limitations": every expert-base offset int64).
 *  - bf16 tensors are passed as uint16_t bit patterns.
 *  - Device faults surface as NF4MOE_ERR_HIP at the caller's next stream
 *    synchronisation; nothing is retried or recovered.
 *
 * Formats (the pages' layouts, "Supported scope" and "The MXFP4 native-byte lane")
 *  NF4_B64   codes uint8 [.., N, K/2], two codes per byte, HIGH nibble = even k;
 *            scales float32 absmax [.., N, K/64]; value = codebook[code] * absmax
 *            rounded once to fp32. K % 64 == 0. The 16 codebook values are the
 *            NormalFloat construction (see nf4moe_codebook).
 *  MXFP4_B32 codes uint8 [.., N, K/2], LOW nibble = even k, OCP e2m1 values;
 *            scales uint8 e8m0 [.., N, K/32]; value = e2m1(code) * 2^(e8m0-127),
 *            e8m0 = 255 is NaN. K % 32 == 0.
 *  NF4_B64_BF16ABS  as NF4_B64 with the absmax stored as bf16 bits, uint16
 *            [.., N, K/64]; the decode widens it to fp32 first.
 */
#ifndef NF4MOE_H
#define NF4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NF4MOE_OK = 0,
  NF4MOE_ERR_INVALID_ARG = 1, /* bad size, null or misaligned pointer, bad enum */
  NF4MOE_ERR_UNSUPPORTED = 2, /* valid request outside what this library supports */
  NF4MOE_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required     */
  NF4MOE_ERR_HIP = 4          /* a HIP runtime call failed (launch, device query) */
} nf4moe_status_t;

/* Weight formats. NF4_B64_BF16ABS is NF4_B64 with each block's absmax stored
 * as bf16 (2 bytes instead of 4, 5.6 % fewer bytes per weight row): the
 * experts4bit-qlora page's bf16 absmax, lossless for bf16-source weights
 * because a block maximum of bf16 values is a bf16 value ("The one ordering
 * trap" paragraph before it: --absmax-dtype bf16). Codes, nibble order and the
 * decode c[code] * absmax (one fp32 product) are those of NF4_B64. */
typedef enum {
  NF4MOE_FMT_NF4_B64 = 0,
  NF4MOE_FMT_MXFP4_B32 = 1,
  NF4MOE_FMT_NF4_B64_BF16ABS = 2
} nf4moe_format_t;
typedef enum { NF4MOE_DT_F32 = 0, NF4MOE_DT_BF16 = 1 } nf4moe_dtype_t;

/* Which grouped-GEMM kernel family runs. AUTO picks from the routed row count
 * known on the host (R = T * top_k): R <= 64 for NF4 and R <= 48 for MXFP4
 * (with H, I <= 4096) runs the bandwidth-bound decode kernels, larger R the
 * MFMA kernels (tiles of up to 64 rows of one expert when the groups average
 * at most 48 rows, else up to 128; each tile runs a 128-, 64- or 32-row body
 * by its row count). The other values force one family (for A/B measurement
 * and tests); the result must satisfy the same tolerance. */
typedef enum { NF4MOE_PATH_AUTO = 0, NF4MOE_PATH_SMALL_M = 1, NF4MOE_PATH_MFMA = 2 } nf4moe_path_t;

/* nf4moe_auto_path -- the family AUTO runs for a grouped GEMM of R routed rows
 * whose K (for a forward: max(H, I)) is K_max, in format fmt: NF4MOE_PATH_SMALL_M
 * or NF4MOE_PATH_MFMA. Host only; no errors. */
int32_t nf4moe_auto_path(nf4moe_format_t fmt, int64_t R, int64_t K_max);

/* The gate_up epilogue. SWIGLU: h = silu(g) * u, silu(g) = g / (1 + exp(-g)).
 * CLAMPED: the gpt-oss expert form the experts4bit-qlora page names without
 * defining it ("Scope": MXFP4 experts with per-expert biases and a clamped-GLU
 * epilogue); read here as g' = min(g, limit), u' = clamp(u, -limit, limit),
 * h = (u' + 1) * g' / (1 + exp(-alpha * g')), alpha and limit given by the
 * caller (gpt-oss publishes alpha = 1.702, limit = 7). */
typedef enum { NF4MOE_GLU_SWIGLU = 0, NF4MOE_GLU_CLAMPED = 1 } nf4moe_glu_t;

/* One MoE layer. All pointers are device memory owned by the caller.
 * The fused gate_up stack is [E, 2I, H] (rows [0, I) gate, [I, 2I) up, or with
 * glu_interleaved rows 2c gate and 2c + 1 up) and the down stack [E, H, I] --
 * the experts4bit-qlora README's fused expert-stack convention ("Quickstart")
 * -- each stored in `fmt`. Optional per-expert biases (the gpt-oss form):
 * b13 [E, 2I] fp32 added to the gate_up product row by row (same row order as
 * w13) before the epilogue, b2 [E, H] fp32 added to each expert's down output
 * before its routing weight. A zero-filled struct tail (glu 0, biases NULL)
 * is the plain SwiGLU layer. */
typedef struct {
  nf4moe_format_t fmt;
  int32_t E;           /* experts, 1..1024                                   */
  int32_t H;           /* hidden size (K of gate_up, N of down)              */
  int32_t I;           /* intermediate size (K of down)                      */
  int32_t top_k;       /* experts per token, 1..min(E, 32)                   */
  int32_t renormalize; /* 1: softmax over the k selected logits; 0: full softmax at the ids */
  int32_t path;        /* nf4moe_path_t                                      */
  const uint8_t *w13;  /* [E, 2I, H/2] codes                                  */
  const void *w13_scale; /* NF4: float [E, 2I, H/64]; MXFP4: uint8 [E, 2I, H/32] */
  const uint8_t *w2;   /* [E, H, I/2] codes                                   */
  const void *w2_scale;  /* NF4: float [E, H, I/64];  MXFP4: uint8 [E, H, I/32]  */
  const float *router_w; /* [E, H] fp32                                        */
  const float *router_b; /* [E] fp32 added to the logits, or NULL              */
  int32_t glu;           /* nf4moe_glu_t                                        */
  float glu_alpha;       /* CLAMPED only: > 0, finite                           */
  float glu_limit;       /* CLAMPED only: > 0, finite                           */
  int32_t glu_interleaved; /* 0: gate rows [0, I), up [I, 2I); 1: gate 2c, up 2c + 1 */
  const float *b13;      /* [E, 2I] fp32 or NULL                                */
  const float *b2;       /* [E, H] fp32 or NULL                                 */
} nf4moe_layer_t;

/* ---------------------------------------------------------------------------
 * nf4moe_quantize -- fp32 weights [rows, K] (device, row-major) -> packed codes
 * [rows, K/2] + scales (device). Off the timed path.
 * NF4 (grouped-nf4-gemm PKG-INFO, "Try it on CPU right now", block 1): absmax =
 *   max |w| over each 64-block, stored fp32; code = the exact nearest codebook
 *   value to w/absmax (decided by fp64 midpoint comparisons), ties to the lower
 *   code; an all-zero block stores absmax 0 and code 7 (0.0).
 * MXFP4 (same section, block 2; OCP MX v1.0): X = floor(log2 amax) - 2 clamped
 *   to [-127, 127], e8m0 = X + 127; code = nearest e2m1 of w / 2^X, ties to the
 *   even code, saturating at 6; code bit 3 = the input's sign bit.
 * NF4_B64_BF16ABS: the NF4 rule with the block absmax rounded up to the nearest
 *   bf16 value before the codes are chosen (no change when it is one, as for
 *   bf16-source weights: then codes and decoded values equal NF4_B64's); scales
 *   uint16 bf16 bits [rows, K/64].
 * Errors: INVALID_ARG for null pointers, rows < 0, K not a multiple of the block,
 * packed not 4-byte aligned. rows == 0 is a no-op. Non-finite inputs give
 * unspecified codes.
 * ------------------------------------------------------------------------- */
nf4moe_status_t nf4moe_quantize(nf4moe_format_t fmt, const float *w, int64_t rows, int64_t K,
                                uint8_t *packed, void *scale, void *stream);

/* nf4moe_dequantize -- packed codes + scales (device) -> fp32 [rows, K] (device).
 * A test export of the decode the GEMM kernels perform in registers: every
 * element equals the reference decode bit for bit ("Expected result": the
 * per-element decode is identical). Errors as for nf4moe_quantize. */
nf4moe_status_t nf4moe_dequantize(nf4moe_format_t fmt, const uint8_t *packed, const void *scale,
                                  int64_t rows, int64_t K, float *w_out, void *stream);

/* nf4moe_absmax_to_bf16 -- the bf16 absmax cast of an existing NF4_B64 scale
 * array (experts4bit-qlora page, the --absmax-dtype bf16 paragraph: the cast is
 * taken only where it is exact and is refused otherwise). absmax fp32 [n] ->
 * out uint16 bf16 bits [n], each rounded up to the nearest bf16 value when it
 * is not one; *n_inexact (device int32, zeroed by the caller) receives the
 * number of such entries: a caller refuses the cast unless it reads 0, and the
 * codes stay valid only then. Asynchronous on `stream`. Errors: INVALID_ARG for
 * n < 0, NULL or misaligned pointers; n == 0 is a no-op. */
nf4moe_status_t nf4moe_absmax_to_bf16(const float *absmax, int64_t n, uint16_t *out, int32_t *n_inexact,
                                      void *stream);

/* nf4moe_router_workspace_bytes -- workspace that lets nf4moe_router_logits use
 * the matrix cores for T tokens (the partial sums over 8 chunks of H: 4 * S * T
 * * E bytes, S = min(8, H / 16)); 0 for T < 1, E < 1, or H not a positive
 * multiple of 16 (the vector path needs none). */
size_t nf4moe_router_workspace_bytes(int32_t T, int32_t E, int32_t H);

/* nf4moe_router_logits -- logits[t, e] = sum_h x[t, h] * router_w[e, h] (+ router_b[e]),
 * x bf16 [T, H], router_w fp32 [E, H], optional router_b fp32 [E], logits fp32
 * [T, E] (all device); fp32-accurate accumulation. The first step of the routed
 * layer (the router, outside the kernel on the pages' "Why it happens" dataflow,
 * inside this library). ws (device, caller-owned, 256-byte aligned) may be NULL.
 * With ws and H % 16 == 0 the product runs on the matrix cores: x exact in
 * bf16, each weight as the exact sum of three bf16 parts (weights of normal
 * range), fp32 partial sums over S chunks of H added in chunk order, then the
 * bias; these are the bits nf4moe_moe_forward routes on when it takes the MFMA
 * path. Without ws: the vector ALUs (one workgroup per expert, a token's sum in
 * the same order for every T, up to 256 tokens; a tiled kernel above). Either
 * way a token's logits carry the same bits whatever the other tokens.
 * Errors: INVALID_ARG for T < 0, E outside 1..1024, H <= 0 or H % 8, null or
 * misaligned pointers; WORKSPACE for a non-NULL ws (H % 16 == 0) smaller than
 * nf4moe_router_workspace_bytes(T, E, H). */
nf4moe_status_t nf4moe_router_logits(const uint16_t *x, int32_t T, int32_t H,
                                     const float *router_w, const float *router_b, int32_t E,
                                     float *logits, void *ws, size_t ws_bytes, void *stream);

/* nf4moe_route_workspace_bytes -- workspace nf4moe_route_permute needs. */
size_t nf4moe_route_workspace_bytes(int32_t T, int32_t E, int32_t top_k);

/* nf4moe_route_permute -- top-k + softmax and grouping by expert, from given fp32
 * logits [T, E] (device). Outputs (device):
 *   topk_ids [T, k] int32: the k largest logits per token, ordered by (logit
 *     descending, expert id ascending);
 *   topk_w [T, k] fp32: renormalize=1 -> exp(L_j - L_0) / sum_j' exp(L_j' - L_0);
 *     renormalize=0 -> softmax over all E at the selected ids;
 *   expert_offsets [E+1] int32: rows of expert e are [off[e], off[e+1]);
 *   sorted_slots [T*k] int32: slots s = t*k + j grouped by expert, ascending s
 *     within an expert (a stable counting sort).
 * This is the pages' "a_cat sorted by expert, sizes + expert_ids" grouping
 * ("Why it happens" dataflow), done on the device with no host sync.
 * ids, offsets and slots are exact integers (bit-identical to a stable sort of
 * the same fp32 logits). Non-finite logits: the order compares IEEE total-order
 * keys with -0 taken as +0 (+inf and -inf in place, a positive NaN above +inf,
 * a negative NaN below -inf; ties still go to the lower id), so every token
 * always gets k distinct experts and every index stays in range; the weights
 * of a token with a NaN or infinite logit are unspecified (NaN in practice).
 * Errors: INVALID_ARG (T < 0, E outside 1..1024, top_k outside 1..min(E, 32),
 * null pointers), WORKSPACE (ws_bytes too small). */
nf4moe_status_t nf4moe_route_permute(const float *logits, int32_t T, int32_t E, int32_t top_k,
                                     int32_t renormalize, int32_t *topk_ids, float *topk_w,
                                     int32_t *expert_offsets, int32_t *sorted_slots,
                                     void *ws, size_t ws_bytes, void *stream);

/* nf4moe_gemm_workspace_bytes -- workspace nf4moe_grouped_gemm needs. */
size_t nf4moe_gemm_workspace_bytes(int32_t G, int32_t R);

/* nf4moe_grouped_gemm -- the pages' gemm_4bit_grouped ("Smallest correct example",
 * "Supported scope"): c[r, :] = a[row(r), :] . W[e(r)]^T over routed groups,
 * W decoded from 4-bit codes in registers, fp32 accumulation.
 *   a        bf16 [a_rows, K] (device, 16-byte aligned rows: K % 8 == 0)
 *   a_row_of int32 [R] (device) or NULL: row r reads a[a_row_of[r]] (gather),
 *            NULL means a[r] (then a_rows >= R). Indices outside [0, a_rows)
 *            are a caller error; the kernels clamp them into that range, so
 *            such a row's output is unspecified but no read leaves a
 *   B, B_scale  expert stack [E, N, K/2] + scales in `fmt` (device)
 *   G, group_offsets int32 [G+1] (device): group g = rows [off[g], off[g+1]),
 *            off[0] = 0, non-decreasing, off[G] = R (the caller guarantees this;
 *            kernels clamp to R so a violation cannot write out of bounds)
 *   group_experts int32 [G] (device) or NULL (group g uses expert g); values in [0, E)
 *   c        [R, N] fp32 or bf16 (RNE) in group order (device)
 *   path     nf4moe_path_t
 * Empty groups are allowed. Errors: INVALID_ARG (K or N not a multiple of the
 * format block / of 64, null pointers, R < 0, G outside 1..65536), WORKSPACE. */
nf4moe_status_t nf4moe_grouped_gemm(nf4moe_format_t fmt, const uint16_t *a, const int32_t *a_row_of,
                                    int32_t a_rows, const uint8_t *B, const void *B_scale, int32_t E,
                                    int64_t N, int64_t K, int32_t G, const int32_t *group_offsets,
                                    const int32_t *group_experts, int32_t R, void *c,
                                    nf4moe_dtype_t c_dtype, int32_t path, void *ws, size_t ws_bytes,
                                    void *stream);

/* nf4moe_grouped_dgrad -- the pages' dgrad_4bit_grouped (grouped-nf4-gemm page,
 * "Training: the backward is a kernel too"): the input gradient of
 * nf4moe_grouped_gemm, da[r, :] = dc[r, :] . W[e(r)] over routed groups, W the
 * [N, K] weights decoded from 4-bit codes exactly as the forward decodes them
 * (never written out), fp32 accumulation.
 *   dc       bf16 [R, N] gradient of the GEMM output, rows in group order (device,
 *            16-byte aligned)
 *   B, B_scale  expert stack [E, N, K/2] + scales in `fmt` (device)
 *   G, group_offsets, group_experts  as nf4moe_grouped_gemm (empty groups allowed)
 *   da       [R, K] fp32 or bf16 (RNE), same row order (device)
 *   ws       nf4moe_gemm_workspace_bytes(G, R) bytes, 256-byte aligned (device)
 * Matrix-core kernel for every R (tiles of 128 rows x 128 columns).
 * Errors: INVALID_ARG (K not a multiple of the format block, bad sizes, null or
 * misaligned pointers), UNSUPPORTED (N % 64 != 0), WORKSPACE. */
nf4moe_status_t nf4moe_grouped_dgrad(nf4moe_format_t fmt, const uint16_t *dc, const uint8_t *B,
                                     const void *B_scale, int32_t E, int64_t N, int64_t K, int32_t G,
                                     const int32_t *group_offsets, const int32_t *group_experts,
                                     int32_t R, void *da, nf4moe_dtype_t da_dtype, void *ws,
                                     size_t ws_bytes, void *stream);

/* nf4moe_workspace_bytes -- workspace nf4moe_moe_forward needs for T <= T_max. */
size_t nf4moe_workspace_bytes(const nf4moe_layer_t *layer, int32_t T_max);

/* nf4moe_moe_forward -- one routed MoE layer: router logits, top-k + softmax,
 * grouping by expert, grouped gate_up GEMM with in-register decode, SwiGLU
 * (silu(gate) * up), grouped down GEMM, and the router-weighted combine
 * out[t] = bf16_RNE( sum_j w[t, j] * y[t*k + j] ) summed in fp32. The pages'
 * moe_layer_forward "gate -> GLU -> down" (grouped-nf4-gemm PKG-INFO, "The NVMe
 * tier") plus the routing and combine the pages leave upstream.
 *   x   bf16 [T, H] (device, 16-byte aligned, H % 64 == 0)
 *   out bf16 [T, H] (device)
 *   topk_ids_out [T, k] int32 / topk_w_out [T, k] fp32: optional copies of the
 *   routing decision (device, may be NULL).
 * The gate_up epilogue is SwiGLU, or with layer->glu the clamped GLU with the
 * layer's biases (see nf4moe_glu_t). Intermediates (h, partial products) stay
 * fp32; no bf16 expert weight is written anywhere.
 * Non-finite input (NaN or inf in x, the weights or the router): routing keeps
 * the order of nf4moe_route_permute (k distinct in-range experts per token,
 * whichever kernel routes), so no index leaves its buffer; the outputs of the
 * affected tokens are then unspecified.
 * Row-count invariance (the pages' STATUS page, kernel section): on the small-M
 * path (AUTO picks it for T * top_k <= 64, 48 for MXFP4) a token's outputs and routing carry
 * the same bits whatever the other tokens of the call, for every T; on the
 * MFMA path, among calls of up to 16 tokens (routed on the vector router's
 * logits) and among calls of more than 16 (the matrix-core router's); across
 * these they differ in summation order.
 * Errors: INVALID_ARG (layer fields, sizes, pointers), WORKSPACE (ws_bytes <
 * nf4moe_workspace_bytes(layer, T)). T == 0 is a no-op. */
nf4moe_status_t nf4moe_moe_forward(const nf4moe_layer_t *layer, const uint16_t *x, int32_t T,
                                   uint16_t *out, int32_t *topk_ids_out, float *topk_w_out,
                                   void *ws, size_t ws_bytes, void *stream);

/* nf4moe_moe_forward_noalloc -- nf4moe_moe_forward for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): no workspace argument; the scratch is a
 * library-owned device array of NF4MOE_NOALLOC_SCRATCH_BYTES (32 MiB) that each
 * GPU the library runs on holds until the process ends, looked up on the
 * first call on that device. The call allocates nothing and uses the scratch
 * of the device current on the calling thread (the stream must belong to it).
 * Same kernels and the same results, bit for bit, as nf4moe_moe_forward with a
 * workspace; nothing in the scratch has to start at zero.
 * Limit: layers and token counts with nf4moe_workspace_bytes(layer, T) <=
 * NF4MOE_NOALLOC_SCRATCH_BYTES (an OLMoE-1B-7B-shaped layer, E=64, top_k=8,
 * H=2048, I=1024, up to 333 tokens); larger calls return WORKSPACE and enqueue
 * nothing.
 * Every call on one GPU shares that GPU's scratch, which keeps the last call's
 * contents: calls on one stream are ordered, but calls that can overlap on one
 * GPU (several streams or threads) race and must be serialised by the caller.
 * The scratch address lookup is a runtime query, not a stream operation; a
 * caller that captures this call into a graph can make one eager call on each
 * device first so that the capture holds kernel launches only.
 * Errors as for nf4moe_moe_forward. */
#define NF4MOE_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
nf4moe_status_t nf4moe_moe_forward_noalloc(const nf4moe_layer_t *layer, const uint16_t *x, int32_t T,
                                           uint16_t *out, int32_t *topk_ids_out, float *topk_w_out,
                                           void *stream);

/* nf4moe_moe_forward_profiled -- nf4moe_moe_forward (same kernels, same result,
 * no topk copies) that also uses six caller-created timing HIP events
 * (hipEvent_t, hipEventDefault flags) on `stream`: events[0] is recorded before
 * the router, events[1] after routing + grouping, events[2] after the gate_up +
 * SwiGLU kernel, events[3] after the down projection and combine; events[4] and
 * events[5] are handed to the gate_up kernel's launch (hipExtLaunchKernelGGL)
 * and so carry that kernel's own start and end times. For measurement. Errors
 * as for nf4moe_moe_forward, plus INVALID_ARG for a NULL events array. */
nf4moe_status_t nf4moe_moe_forward_profiled(const nf4moe_layer_t *layer, const uint16_t *x,
                                            int32_t T, uint16_t *out, void *ws, size_t ws_bytes,
                                            void *stream, void *const *events);

/* ---------------------------------------------------------------------------
 * Fine-tuning and multi-adapter serving around the frozen 4-bit layer. These
 * calls follow the same conventions (caller-owned device memory, checks before
 * anything is enqueued, one stream, no host synchronisation, capturable). An
 * output (or workspace) overlaps neither an input nor another output, except where
 * a call says that it may be one: INVALID_ARG otherwise.
 *
 * 8-bit activation checkpoints. A tensor [rows, K] kept for the backward pass as
 * one byte per value and one e8m0 scale byte b per 32 consecutive k (multiplier
 * 2^(b - 127)), the OCP MX v1.0 element formats:
 *   MXINT8  X = floor(log2 amax); code int8 = RNE(v / 2^(X - 6)) in [-127, 127]
 *   MXFP8   X = floor(log2 amax) - 8; code = e4m3 RNE(v / 2^X), saturated at 448
 * X at least -127, b = X + 127. Every code is an exact function of the input
 * (power-of-two scale, ties to even) and every decoded value is exact in bf16
 * where bf16 has the range. A block holding a NaN or an infinity gets b = 255
 * and decodes to NaN as a whole. K % 32 == 0; any alignment of codes and scale.
 * ------------------------------------------------------------------------- */
typedef enum { NF4MOE_CKPT_MXINT8 = 0, NF4MOE_CKPT_MXFP8 = 1 } nf4moe_ckpt8_t;

/* How a tensor that the backward reads is held: as values, or as a checkpoint
 * (codes, with the scales beside them). */
typedef enum {
  NF4MOE_SRC_F32 = 0,
  NF4MOE_SRC_BF16 = 1,
  NF4MOE_SRC_MXINT8 = 2,
  NF4MOE_SRC_MXFP8 = 3
} nf4moe_src_t;

/* nf4moe_ckpt8_quantize / _dequantize -- x fp32 or bf16 [rows, K] -> codes uint8
 * [rows, K], scale uint8 [rows, K/32], and back to fp32 or bf16. rows == 0 is a
 * no-op. Errors: INVALID_ARG (format, dtype, rows < 0, K not a positive multiple
 * of 32, null pointers, x or out not aligned to its element). */
nf4moe_status_t nf4moe_ckpt8_quantize(nf4moe_ckpt8_t fmt, const void *x, nf4moe_dtype_t x_dtype, int64_t rows, int64_t K,
                                      uint8_t *codes, uint8_t *scale, void *stream);
nf4moe_status_t nf4moe_ckpt8_dequantize(nf4moe_ckpt8_t fmt, const uint8_t *codes, const uint8_t *scale, int64_t rows,
                                        int64_t K, void *out, nf4moe_dtype_t out_dtype, void *stream);

/* nf4moe_glu_forward -- h[r] = the gated activation (nf4moe_glu_t) of the gate_up
 * product gu [R, 2I] (fp32 or bf16; gate and up in halves, or interleaved as in
 * nf4moe_layer_t), bf16 RNE [R, I]. With codes / scale the same pass also writes
 * gu's 8-bit checkpoint ([R, 2I] and [R, 2I/32], format ckpt); both NULL saves
 * nothing. I % 32 == 0. R == 0 is a no-op. Errors: INVALID_ARG; UNSUPPORTED for I
 * past 2^30 or R * I past 2^36. */
nf4moe_status_t nf4moe_glu_forward(const void *gu, nf4moe_dtype_t gu_dtype, int64_t R, int32_t I, int32_t glu,
                                   float glu_alpha, float glu_limit, int32_t glu_interleaved, uint16_t *h,
                                   nf4moe_ckpt8_t ckpt, uint8_t *codes, uint8_t *scale, void *stream);

/* nf4moe_glu_backward -- gradient of nf4moe_glu_forward at the gu that is held
 * (gu_src: values, or a checkpoint decoded in registers; gu_scale only for a
 * checkpoint). dh [R, I] is the gradient of h for a row weight of 1 (fp32 or
 * bf16); row_w fp32 [R] (NULL: 1) scales each row's gradient, as the router's
 * weight scales an expert's output:
 *   dgu    bf16 [R, 2I]   row_w[r] * dh[r] through the activation, in gu's layout
 *   h      bf16 [R, I]    the activation recomputed (optional)
 *   drow_w fp32 [R]       sum_c dh[r, c] * h[r, c], the gradient of row_w (optional)
 * The clamped form's gradient is that of the unclamped side at the limit itself.
 * Errors: INVALID_ARG, UNSUPPORTED as for the forward. */
nf4moe_status_t nf4moe_glu_backward(const void *dh, nf4moe_dtype_t dh_dtype, nf4moe_src_t gu_src, const void *gu,
                                    const uint8_t *gu_scale, int64_t R, int32_t I, int32_t glu, float glu_alpha,
                                    float glu_limit, int32_t glu_interleaved, const float *row_w, uint16_t *dgu,
                                    uint16_t *h, float *drow_w, void *stream);

/* ---------------------------------------------------------------------------
 * The norms around a block, fused with its gate and residual scale. Row by row
 * over [T, H], with the residual stream x, the block's output f and, where the
 * next block has one, its pre norm:
 *   z  = f * rstd_post * w_post      rstd_post = 1 / sqrt(mean(f^2) + eps); z = f
 *                                    without w_post
 *   x' = x + alpha * phi(gate) * z   stored as x_dtype, one rounding
 *   y  = x' * rstd_pre * w_pre       of the stored x', bf16
 * One pass; fp32 in registers. gate: none, one value per channel [H], per row
 * [T], or per element [T, H] (fp32 or bf16); phi the identity, sigmoid or tanh.
 * f NULL: a pre norm alone (x is left where it is). w_pre NULL: no pre norm.
 * H is 1..16384; rows are contiguous; no alignment beyond the element's.
 * ------------------------------------------------------------------------- */
typedef enum { NF4MOE_GATE_NONE = 0, NF4MOE_GATE_CHANNEL = 1, NF4MOE_GATE_ROW = 2, NF4MOE_GATE_FULL = 3 } nf4moe_gate_kind_t;
typedef enum { NF4MOE_GATE_IDENTITY = 0, NF4MOE_GATE_SIGMOID = 1, NF4MOE_GATE_TANH = 2 } nf4moe_gate_fn_t;

typedef struct {
  int32_t H;
  int32_t x_dtype;       /* nf4moe_dtype_t of x, x', dx', dx                   */
  const float *w_post;   /* [H] or NULL                                        */
  const float *w_pre;    /* [H] or NULL                                        */
  const void *gate;      /* by gate_kind; NULL with NF4MOE_GATE_NONE           */
  int32_t gate_kind;     /* nf4moe_gate_kind_t                                 */
  int32_t gate_dtype;    /* nf4moe_dtype_t                                     */
  int32_t gate_fn;       /* nf4moe_gate_fn_t                                   */
  float alpha;           /* residual scale, finite                             */
  float eps;             /* finite, >= 0                                       */
} nf4moe_block_norm_t;

/* nf4moe_block_norm_forward -- x [T, H], f bf16 [T, H] or NULL -> x_new [T, H]
 * (may be x itself; not written without f), y bf16 [T, H] (with w_pre),
 * rstd_post / rstd_pre fp32 [T] (with w_post / w_pre; the backward reads them).
 * T == 0 is a no-op. Errors: INVALID_ARG. */
nf4moe_status_t nf4moe_block_norm_forward(const nf4moe_block_norm_t *norm, const void *x, const uint16_t *f, int64_t T,
                                          void *x_new, uint16_t *y, float *rstd_post, float *rstd_pre, void *stream);

/* nf4moe_block_norm_workspace_bytes -- workspace of the backward (0 for T < 1). */
size_t nf4moe_block_norm_workspace_bytes(int32_t H, int64_t T);

/* nf4moe_block_norm_backward -- gradients of the forward from dx_new (of x', in
 * x_dtype; NULL: zero) and dy (of y, bf16; with w_pre), with what the forward
 * read and returned (x_new: the stored x'; without f, x):
 *   dx in x_dtype; df bf16 (with f); dgate fp32 in the gate's shape; dw_post,
 *   dw_pre fp32 [H]. Sums over rows are added in a fixed order (the same bits on
 *   every run). T == 0 writes zeros to dw_post, dw_pre and a per-channel dgate.
 * Errors: INVALID_ARG, WORKSPACE. */
nf4moe_status_t nf4moe_block_norm_backward(const nf4moe_block_norm_t *norm, const void *dx_new, const uint16_t *dy,
                                           const void *x_new, const uint16_t *f, const float *rstd_post,
                                           const float *rstd_pre, int64_t T, void *dx, uint16_t *df, float *dgate,
                                           float *dw_post, float *dw_pre, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests or experts beside a shared projection (the
 * frozen 4-bit one of nf4moe_grouped_gemm, or any other). Row r of R has adapter
 * l = ids[r]; an id outside [0, L) means none:
 *   t[r]   = A_l x[x_row_of[r]]                 fp32
 *   out[r] = base[r] + scale_l * B_l t[r]       one rounding; rows without an
 *                                               adapter: base[r]
 * Rows may come in any order; one adapter per expert is ids = the rows' experts,
 * one per (request, expert) an id that counts both. A NaN or an infinity reaches
 * the values that are computed from it and no others; those are then not finite
 * (NaN where the plain formula may have an infinity: the fp32 low-rank values are
 * multiplied as three exact parts).
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t L;           /* adapters, 1..4096                                    */
  int32_t rank;        /* a multiple of 8 in 8..128 (pad smaller ones with 0)  */
  int32_t K, N;        /* input and output width, multiples of 8, at most 2^20 */
  const uint16_t *A;   /* bf16 [L, rank, K]                                    */
  const uint16_t *B;   /* bf16 [L, N, rank]                                    */
  const float *scale;  /* fp32 [L], or NULL: 1                                 */
} nf4moe_adapters_t;

/* nf4moe_adapter_plan -- the grouping of ids [R] (device) by adapter, which the
 * calls below otherwise make for themselves: a batch that runs through several
 * projections builds it once. plan: nf4moe_adapter_plan_bytes(R, L) bytes, device,
 * 256-byte aligned; it holds for these ids, R and L only. R at most 2^30; R == 0
 * is a no-op. Errors: INVALID_ARG, WORKSPACE. */
size_t nf4moe_adapter_plan_bytes(int32_t R, int32_t L);
nf4moe_status_t nf4moe_adapter_plan(const int32_t *ids, int32_t R, int32_t L, void *plan, size_t plan_bytes, void *stream);

/* nf4moe_adapter_workspace_bytes -- workspace of the forward (backward = 0) or the
 * backward (1) for R rows; 0 for invalid sizes or R < 1, and where the forward
 * needs none (its one-launch form). */
size_t nf4moe_adapter_workspace_bytes(const nf4moe_adapters_t *ad, int32_t R, int32_t backward);

/* nf4moe_adapter_forward -- out [R, N] (may be base) from x bf16 [x_rows, K] and
 * base [R, N] or NULL (zeros), both in dtype.
 *   x_row_of int32 [R] (device) or NULL: row r reads x[x_row_of[r]], clamped into
 *            [0, x_rows); NULL means x[r] (then x_rows >= R)
 *   plan     from nf4moe_adapter_plan for the same ids, or NULL
 *   t        fp32 [R, rank] (16-byte aligned) or NULL: the low-rank product, which
 *            the backward takes (0 for rows without an adapter)
 * t is summed in fp32 and enters the second product exactly; the output has one
 * rounding. R == 0 is a no-op. Calls that need no workspace (few rows for their
 * rank and widths) run in one launch and ignore the plan; results differ from the
 * grouped kernels' in summation order only. Errors: INVALID_ARG, WORKSPACE,
 * UNSUPPORTED where a launch would pass 2^32 threads. */
nf4moe_status_t nf4moe_adapter_forward(const nf4moe_adapters_t *ad, const uint16_t *x, int32_t x_rows,
                                       const int32_t *x_row_of, const int32_t *ids, const void *plan, size_t plan_bytes,
                                       int32_t R, const void *base, void *out, nf4moe_dtype_t dtype, float *t, void *ws,
                                       size_t ws_bytes, void *stream);

/* nf4moe_adapter_backward -- for dy bf16 [R, N], the gradient of out:
 *   u[r] = scale_l * B_l^T dy[r]                                  (kept in fp32)
 *   dx[r] = dx_base[r] + A_l^T u[r]    [R, K] in dx_dtype; dx_base NULL: zeros, may
 *                                      be dx; rows without an adapter: dx_base[r].
 *                                      Per routed row, as nf4moe_grouped_dgrad
 *   dA_l = sum_r u[r] x[x_row_of[r]]^T    fp32 [L, rank, K]
 *   dB_l = scale_l * sum_r dy[r] t[r]^T   fp32 [L, N, rank]
 * over the rows of adapter l, zeros for an adapter without rows whatever its scale; the
 * weights of all L adapters are read, used or not (for dx, dA). dx, dA and dB may
 * each be NULL. x (with x_rows) is read for dA only: bf16, or an 8-bit checkpoint
 * (x_src, with x_scale; K % 32 == 0) decoded in registers. t is the forward's (for
 * dB). The sums over rows are added in a fixed order: the same bits on every run. dA
 * and dB 16-byte aligned. R == 0 writes zeros to dA and dB. Errors: INVALID_ARG,
 * WORKSPACE, UNSUPPORTED where a launch would pass 2^32 threads. */
nf4moe_status_t nf4moe_adapter_backward(const nf4moe_adapters_t *ad, const uint16_t *dy, nf4moe_src_t x_src, const void *x,
                                        const uint8_t *x_scale, int32_t x_rows, const int32_t *x_row_of, const float *t,
                                        const int32_t *ids, const void *plan, size_t plan_bytes, int32_t R,
                                        const void *dx_base, void *dx, nf4moe_dtype_t dx_dtype, float *dA, float *dB,
                                        void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The dense bf16 ends of a training step around the frozen layer: a gated feed-forward's gate
 * and up half (of a shared expert; the down projection is the caller's), the losses of a
 * vocabulary head, layer norm. The conventions are those of the fine-tuning calls above. Matrices
 * are bf16, contiguous and 16-byte aligned, their widths (H, I) multiples of 8 up to 2^20;
 * products are summed in fp32, every output is rounded once; the gradient of a product (dgu, P below) is rounded to bf16 where it becomes
 * an operand of the next, up to 64 rows to the sum of two bf16 values, P of more rows without a
 * factor that their dloss have in common (1 / rows of a mean loss, say, is not rounded). The same bits on every run of
 * the same call (dx asked for without the weight's gradient may be summed in another order than
 * beside it). UNSUPPORTED past 2^22 tiles of 256 x 256 of one product, 2^38 values, or 2^25 rows of
 * a vocabulary loss.
 *
 * Gated feed-forward: g = x Wg^T, u = x Wu^T, h = the gated activation (nf4moe_glu_t) of g and u.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t H, I;
  const uint16_t *w13;       /* bf16 [2I, H]: gate rows, then up rows; or interleaved */
  int32_t glu;               /* nf4moe_glu_t                                        */
  float glu_alpha, glu_limit;
  int32_t glu_interleaved;   /* rows alternate gate, up (as in nf4moe_layer_t)      */
} nf4moe_gated_ffn_t;

/* nf4moe_gated_ffn_forward -- h bf16 [T, I] from x bf16 [T, H]. One launch, no workspace.
 * T at most 2^30; T == 0 is a no-op. Errors: INVALID_ARG, UNSUPPORTED. */
nf4moe_status_t nf4moe_gated_ffn_forward(const nf4moe_gated_ffn_t *ffn, const uint16_t *x, int64_t T, uint16_t *h,
                                         void *stream);

/* nf4moe_gated_ffn_workspace_bytes -- workspace of the backward (0 for T < 1 or invalid sizes), whatever outputs are
 * asked for: dgu [T, 2I]; up to 64 rows twice that and x, and dx twice in fp32; and where sums are cut into slices
 * fp32 parts of dx and of dw13, at most 64 MB each. */
size_t nf4moe_gated_ffn_workspace_bytes(const nf4moe_gated_ffn_t *ffn, int64_t T);

/* nf4moe_gated_ffn_backward -- gradients for dh bf16 [T, I], g and u computed again:
 *   dx   bf16 [T, H]    dgu W13           (NULL: not computed)
 *   dw13 bf16 [2I, H]   dgu^T x, in w13's row order   (NULL: not computed)
 *   h    bf16 [T, I]    the forward's output again (optional)
 * The clamped form's gradient is that of the unclamped side at the limit itself; a NaN passes through
 * its clamps. T == 0 writes zeros to dw13. Errors: INVALID_ARG (neither dx nor dw13 among them), WORKSPACE, UNSUPPORTED. */
nf4moe_status_t nf4moe_gated_ffn_backward(const nf4moe_gated_ffn_t *ffn, const uint16_t *dh, const uint16_t *x, int64_t T,
                                          uint16_t *dx, uint16_t *dw13, uint16_t *h, void *ws, size_t ws_bytes,
                                          void *stream);

/* The head of the losses below: logits l = x W^T [T, V], never stored. */
typedef struct {
  int32_t H;
  int32_t V;                 /* 1..2^21                                             */
  const uint16_t *w;         /* bf16 [V, H]                                         */
} nf4moe_head_t;

/* nf4moe_vocab_workspace_bytes -- workspace of the forward (backward = 0) or the backward (1) of
 * the cross entropy (k = 0) or of the distillation from k entries a row, for T rows; 0 for T < 1 or
 * invalid sizes. The backward's, whatever outputs are asked for, holds the gradient P of one piece of the vocabulary at
 * a time, at most 128 MB of it, or 256 columns; dx in fp32 where the vocabulary has several pieces, up to 64 rows dx and
 * x twice; and where sums are cut into slices fp32 parts of dx and of a piece of dw, at most 64 MB each. */
size_t nf4moe_vocab_workspace_bytes(const nf4moe_head_t *head, int64_t T, int32_t k, int32_t backward);

/* nf4moe_vocab_ce_forward -- softmax cross entropy: lse[t] = log sum_v exp(l[t, v]) and loss[t] =
 * lse[t] - l[t, labels[t]], fp32 [T]; a label outside [0, V) (-100, say) means loss 0 and no
 * gradient. T == 0 is a no-op. Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED.
 *
 * nf4moe_vocab_ce_backward -- for dloss fp32 [T] (the gradient of loss; where a row has no label it may
 * hold anything) and the forward's lse, with P = dloss (softmax(l) - onehot(label)):
 *   dx bf16 [T, H] = P W;  dw bf16 [V, H] = P^T x     (either may be NULL)
 * A row without a label counts for nothing whatever its x holds. T == 0 writes zeros to dw. */
nf4moe_status_t nf4moe_vocab_ce_forward(const nf4moe_head_t *head, const uint16_t *x, int64_t T, const int32_t *labels,
                                        float *loss, float *lse, void *ws, size_t ws_bytes, void *stream);
nf4moe_status_t nf4moe_vocab_ce_backward(const nf4moe_head_t *head, const float *dloss, const uint16_t *x, int64_t T,
                                         const int32_t *labels, const float *lse, uint16_t *dx, uint16_t *dw, void *ws,
                                         size_t ws_bytes, void *stream);

/* nf4moe_vocab_distill_forward -- distillation from a teacher's top logits: ids int32 [T, k] and the
 * teacher's logits for them (fp32 or bf16 [T, k], k 1..1024), temperature tau in 0.001..1000:
 *   q      fp32 [T, k]  softmax over a row's entries of teacher / tau
 *   logits fp32 [T, k]  the student's logits l[t, ids[t, j]]
 *   lse    fp32 [T]     log sum_v exp(l[t, v] / tau)
 *   loss   fp32 [T]     tau^2 sum_j q_j (log q_j - logits_j / tau + lse), tau^2 times the divergence of
 *                       the student's whole softmax from the teacher's
 * An entry with an id outside [0, V) counts for nothing, whatever its logit (q and logits 0). An id
 * that a row names twice has the sum of both probabilities, in its first place. A row without an
 * entry whose teacher logit is above -inf has loss 0, lse +inf and no gradient. T == 0 is a no-op.
 * Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED.
 *
 * nf4moe_vocab_distill_backward -- with the forward's q, logits and lse, P = dloss tau (softmax(l / tau)
 * - q); dx, dw and the rest as in nf4moe_vocab_ce_backward. */
nf4moe_status_t nf4moe_vocab_distill_forward(const nf4moe_head_t *head, const uint16_t *x, int64_t T, const int32_t *ids,
                                             const void *teacher, nf4moe_dtype_t teacher_dtype, int32_t k,
                                             float temperature, float *loss, float *lse, float *q, float *logits, void *ws,
                                             size_t ws_bytes, void *stream);
nf4moe_status_t nf4moe_vocab_distill_backward(const nf4moe_head_t *head, const float *dloss, const uint16_t *x, int64_t T,
                                              const int32_t *ids, const float *q, const float *logits, const float *lse,
                                              int32_t k, float temperature, uint16_t *dx, uint16_t *dw, void *ws,
                                              size_t ws_bytes, void *stream);

/* Layer norm: y = (x - mean) rstd w + b, rstd = 1 / sqrt(mean((x - mean)^2) + eps), fp32 in
 * registers. Rows contiguous, H 1..16384, no alignment beyond the element's. */
typedef struct {
  int32_t H;
  int32_t x_dtype;           /* nf4moe_dtype_t of x, dx_base, dx                    */
  int32_t y_dtype;           /* ... of y, dy                                        */
  const float *w, *b;        /* fp32 [H] or NULL (1, 0)                             */
  float eps;                 /* finite, >= 0                                        */
} nf4moe_layer_norm_t;

/* nf4moe_layer_norm_forward -- x [T, H] -> y [T, H], mean and rstd fp32 [T] (which the backward
 * reads). T == 0 is a no-op. Errors: INVALID_ARG. */
nf4moe_status_t nf4moe_layer_norm_forward(const nf4moe_layer_norm_t *norm, const void *x, int64_t T, void *y, float *mean,
                                          float *rstd, void *stream);

/* nf4moe_layer_norm_workspace_bytes -- workspace of the backward (0 for T < 1). */
size_t nf4moe_layer_norm_workspace_bytes(int32_t H, int64_t T);

/* nf4moe_layer_norm_backward -- for dy [T, H], with n = (x - mean) rstd and a = dy w:
 *   dx [T, H] = dx_base + rstd (a - mean(a) - n mean(a n))   (dx_base NULL: zero; may be dx)
 *   dw fp32 [H] = sum_t dy n;  db fp32 [H] = sum_t dy
 * dx, dw, db may each be NULL. T == 0 writes zeros to dw and db. Errors: INVALID_ARG, WORKSPACE. */
nf4moe_status_t nf4moe_layer_norm_backward(const nf4moe_layer_norm_t *norm, const void *dy, const void *x, const float *mean,
                                           const float *rstd, int64_t T, const void *dx_base, void *dx, float *dw, float *db,
                                           void *ws, size_t ws_bytes, void *stream);

/* nf4moe_stream_read -- a measurement aid, not part of the layer: one launch
 * that reads `bytes` bytes of `buf` (device, 16-byte aligned, bytes a positive
 * multiple of 16) once with 16-byte loads, loads_per_thread (1, 2, 4, 8 or 16)
 * of them per thread of 256-thread workgroups, and writes one 32-bit XOR per
 * workgroup to sink (device, nf4moe_stream_read_sink_words(bytes,
 * loads_per_thread) words). Its duration gives the plain HBM read rate of a
 * single launch of that size, the measured ceiling the decode kernels are set
 * beside. Errors: INVALID_ARG for a bad size or loads_per_thread, NULL or
 * misaligned pointers; UNSUPPORTED past 2^31 workgroups. */
int64_t nf4moe_stream_read_sink_words(int64_t bytes, int32_t loads_per_thread);
nf4moe_status_t nf4moe_stream_read(const void *buf, int64_t bytes, int32_t loads_per_thread, uint32_t *sink,
                                   void *stream);

/* nf4moe_mfma_peak -- a measurement aid, not part of the layer: one launch of
 * `workgroups` 512-thread workgroups in which every wave runs `iters` rounds of
 * 8 independent bf16 MFMAs (32x32x16) on pseudo-random finite register
 * operands, with no memory traffic; each thread writes one float to sink
 * (device, workgroups * 512 floats). nf4moe_mfma_peak_flops(workgroups,
 * iters) gives the launch's flops (0 for invalid arguments); flops over the
 * launch's duration is the bf16 matrix-core rate the GPU sustains under full
 * load, the measured ceiling beside the published dense peak. Errors:
 * INVALID_ARG for workgroups outside 1..2^20, iters <= 0, a NULL or misaligned
 * sink. */
int64_t nf4moe_mfma_peak_flops(int32_t workgroups, int32_t iters);
nf4moe_status_t nf4moe_mfma_peak(int32_t workgroups, int32_t iters, float *sink, void *stream);

/* nf4moe_codebook -- host copy of the 16 fp32 decode values the kernels use for
 * `fmt` (index = 4-bit code). No device access. Returns INVALID_ARG for a bad fmt
 * or NULL out. */
nf4moe_status_t nf4moe_codebook(nf4moe_format_t fmt, float out[16]);

/* Human-readable name of a status; never NULL. */
const char *nf4moe_status_string(nf4moe_status_t st);

/* Thread-local description of this thread's last non-OK status ("" if none). */
const char *nf4moe_last_error(void);

/* Library version string. */
const char *nf4moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NF4MOE_H */
