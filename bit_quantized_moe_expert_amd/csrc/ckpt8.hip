// 8-bit activation checkpoints (formats in ckpt8.h) and the gated activation
// that writes and reads them.
//
// All of it is bound by memory traffic: every element is read once, worked on in
// registers and written once, 8 elements a thread (16-byte accesses of bf16), at the
// rate of a plain copy or better: see each kernel.
#include "ckpt8.h"
#include "internal.h"
#include "train.h"

namespace nf4moe {

namespace {

// One thread per 8 elements; the 4 threads of a block of 32 share its maximum
// by two lane permutes. n is a multiple of 32, so a block is whole or absent. 8191 x
// 2880 fp32 (119 MB with the codes) 19.4 us to 8 bits and 19.9 back, 6.1 TB/s (the
// last-level cache holds a part); 65 x 2048 bf16 2.5 us, a launch's latency.
template <int FMT, bool BF>
__global__ __launch_bounds__(256) void k_ckpt8_quant(const void *__restrict__ x, int64_t n8, uint8_t *__restrict__ codes,
                                                     uint8_t *__restrict__ scale) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  load_elems8<BF>(x, 8 * i, v);
  const uint32_t b = ckpt8_scale<FMT>(lanes_max_u32<4>(abs_bits_max8(v)));
  store8(codes + 8 * i, ckpt8_encode8<FMT>(v, b));
  if ((i & 3) == 0) scale[i >> 2] = (uint8_t)b;
}

template <int FMT, bool BF>
__global__ __launch_bounds__(256) void k_ckpt8_dequant(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scale,
                                                       int64_t n8, void *__restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  ckpt8_decode8<FMT>(load8(codes + 8 * i), scale[i >> 2], v);
  store_elems8<BF>(out, 8 * i, v);
}

// Gate and up of 8 neighbouring columns of one row, and back. Halves: columns
// c .. c + 7 and I + c ..; interleaved: 16 neighbouring values, gate at the even
// ones.
template <bool BF>
__device__ inline void load_pairs(const void *gu, int64_t row, int I, int inter, int c, float (&g)[8], float (&u)[8]) {
  const int64_t base = row * 2 * I;
  float a[8], b[8];
  load_elems8<BF>(gu, base + (inter ? 2 * c : c), a);
  load_elems8<BF>(gu, base + (inter ? 2 * c + 8 : I + c), b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = inter ? (i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)]) : a[i];
    u[i] = inter ? (i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1]) : b[i];
  }
}
__device__ inline void store_pairs_bf16(uint16_t *dgu, int64_t row, int I, int inter, int c, const float (&g)[8],
                                        const float (&u)[8]) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = inter ? ((i & 1) ? u[i >> 1] : g[i >> 1]) : g[i];
    b[i] = inter ? ((i & 1) ? u[4 + (i >> 1)] : g[4 + (i >> 1)]) : u[i];
  }
  const int64_t base = row * 2 * I;
  store_elems8<true>(dgu, base + (inter ? 2 * c : c), a);
  store_elems8<true>(dgu, base + (inter ? 2 * c + 8 : I + c), b);
}

// The clamped form's g' and u'. Comparisons, so that a NaN (a checkpoint block
// that held one decodes to NaN) stays a NaN in the result.
__device__ inline float clamp_gate(float g, float limit) { return g > limit ? limit : g; }
__device__ inline float clamp_up(float u, float limit) { return u > limit ? limit : (u < -limit ? -limit : u); }

// h = act(gate) * up in bf16, and optionally the 8-bit save of gate and up. One
// thread per 8 columns of a row: the flat index splits into (row, column) by the
// workgroup's first index, once per workgroup. A block of 32 values is 4 threads
// of one half, or 2 threads of interleaved pairs. 32768 x 1024 pairs of bf16 with the
// save: 270 MB in 42 us, 6.4 TB/s (in part the last-level cache). gu is read past the caches, which keep room for h and
// the save: between a kernel that makes gu and one that reads h, us for the three, 129
// -> 114; 8192 x 2880 86 -> 80, 2048 x 2880 the same 24. (Storing past them too gains 4 us
// more there, and costs 8 where the save is read back soon.)
template <bool BF, int FMT>
__global__ __launch_bounds__(256) void k_glu_forward(GluArgs p) {
  const uint32_t I8 = (uint32_t)p.I / 8;
  const int64_t first = (int64_t)blockIdx.x * 256;
  const uint32_t off = (uint32_t)(first % I8) + threadIdx.x;
  const int64_t row = first / I8 + off / I8;
  if (row >= p.R) return;  // whole rows, so whole blocks of 32, leave together
  const int c = 8 * (int)(off % I8);
  const int64_t base = row * 2 * p.I;
  float a[8], b[8];        // the two 8-element pieces as they lie in memory
  load_elems8<BF, true>(p.gu, base + (p.inter ? 2 * c : c), a);
  load_elems8<BF, true>(p.gu, base + (p.inter ? 2 * c + 8 : p.I + c), b);
  float h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = p.inter ? (i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)]) : a[i];
    const float u = p.inter ? (i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1]) : b[i];
    h[i] = p.glu == 1 ? (clamp_up(u, p.limit) + 1.0f) * sig_gate(clamp_gate(g, p.limit), p.alpha) : sig_gate(g, 1.0f) * u;
  }
  store_elems8<true>(p.h, row * p.I + c, h);
  if constexpr (FMT != CK_NONE) {
    const uint32_t ma = abs_bits_max8(a), mb = abs_bits_max8(b);
    uint8_t *q = p.codes + base, *s = p.scale + base / 32;
    if (p.inter) {
      const uint32_t e = ckpt8_scale<FMT>(lanes_max_u32<2>(ma > mb ? ma : mb));
      const uint2 x = ckpt8_encode8<FMT>(a, e), y = ckpt8_encode8<FMT>(b, e);
      store16(q + 2 * c, make_uint4(x.x, x.y, y.x, y.y));
      if ((c & 8) == 0) s[c / 16] = (uint8_t)e;
    } else {
      const uint32_t ea = ckpt8_scale<FMT>(lanes_max_u32<4>(ma)), eb = ckpt8_scale<FMT>(lanes_max_u32<4>(mb));
      store8(q + c, ckpt8_encode8<FMT>(a, ea));
      store8(q + p.I + c, ckpt8_encode8<FMT>(b, eb));
      if ((c & 24) == 0) {
        s[c / 32] = (uint8_t)ea;
        s[(p.I + c) / 32] = (uint8_t)eb;
      }
    }
  }
}

// Backward of the gated activation: with d = row_w * dh, s = sigma(a g'),
//   SwiGLU   dg = d u s (1 + g (1 - s)),              du = d g s,  h = g s u
//   clamped  dg = [g <= limit] d (u' + 1) s (1 + a g' (1 - s)),
//            du = [|u| <= limit] d g' s,              h = (u' + 1) g' s
// and drow = sum_c dh h, the gradient of the row's weight. gate and up come
// from the 8-bit save (decoded here, never written out) or from bf16 / fp32.
// WPR waves per row; drow is their sums added in a fixed order. 32768 x 1024 pairs from
// 8 bits, h recomputed: 337 MB in 54 us, 6.3 TB/s right after the forward (in part the
// last-level cache), 61 from other inputs; with fp32 dh 405 MB in 74, from bf16 gu 403 in 72.
template <int SRC, bool DHBF, int WPR>
__global__ __launch_bounds__(256) void k_glu_backward(GluArgs p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = WPR == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (row >= p.R) return;
  const int I = p.I, inter = p.inter;
  const float w = p.row_w ? p.row_w[row] : 1.0f;
  const float al = p.glu == 1 ? p.alpha : 1.0f;
  float dot = 0.0f;
  for (int c = 8 * (WPR == 4 ? (int)threadIdx.x : lane); c < I; c += 512 * WPR) {
    float g[8], u[8], dh[8];
    if constexpr (SRC == SRC_BF16 || SRC == SRC_F32) {
      load_pairs<SRC == SRC_BF16>(p.gu, row, I, inter, c, g, u);
    } else {
      constexpr int F = SRC - SRC_MXINT8;
      const uint8_t *q = reinterpret_cast<const uint8_t *>(p.gu) + row * 2 * I;
      const uint8_t *s = p.gu_scale + row * 2 * I / 32;
      if (inter) {
        float a[8], b[8];
        const uint4 x = load16(q + 2 * c);
        const uint32_t e = s[c / 16];
        ckpt8_decode8<F>(make_uint2(x.x, x.y), e, a);
        ckpt8_decode8<F>(make_uint2(x.z, x.w), e, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = a[2 * i], u[i] = a[2 * i + 1];
          g[4 + i] = b[2 * i], u[4 + i] = b[2 * i + 1];
        }
      } else {
        const uint2 x = load8(q + c), y = load8(q + I + c);
        ckpt8_decode8<F>(x, s[c / 32], g);
        ckpt8_decode8<F>(y, s[(I + c) / 32], u);
      }
    }
    load_elems8<DHBF>(p.dh, row * I + c, dh);
    float dg[8], du[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float gg = g[i], uu = u[i];
      bool live_g = true, live_u = true;
      if (p.glu == 1) {
        live_g = !(gg > p.limit);
        live_u = !(fabsf(uu) > p.limit);
        gg = clamp_gate(gg, p.limit);
        uu = clamp_up(uu, p.limit) + 1.0f;
      }
      // sigma by the hardware exp2 and reciprocal (about 1 ulp each), as in the
      // forward's epilogue
      const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gg * (-1.44269504088896341f * al)));
      const float gs = gg * sg, d = dh[i] * w;
      h[i] = gs * uu;
      dot += dh[i] * h[i];
      dg[i] = live_g ? d * uu * sg * (1.0f + al * gg * (1.0f - sg)) : 0.0f;
      du[i] = live_u ? d * gs : 0.0f;
    }
    store_pairs_bf16(p.dgu, row, I, inter, c, dg, du);
    if (p.h) store_elems8<true>(p.h, row * I + c, h);
  }
  if (p.drow) {
    dot = wave_sum(dot);
    if constexpr (WPR == 4) {
      __shared__ float part[4];
      if (lane == 0) part[wave] = dot;
      lds_barrier();
      dot = part[0] + part[1] + part[2] + part[3];
      if (threadIdx.x == 0) p.drow[row] = dot;
    } else {
      if (lane == 0) p.drow[row] = dot;
    }
  }
}

// Pieces of at most 2^31 elements keep every grid inside a dispatch's limits.
constexpr int64_t kPiece8 = int64_t(1) << 28;  // threads (8 elements each) per launch, a multiple of 256

}  // namespace

hipError_t launch_ckpt8_quantize(int fmt, const void *x, bool x_bf16, int64_t n, uint8_t *codes, uint8_t *scale,
                                 hipStream_t s) {
  for (int64_t t0 = 0; t0 < n / 8; t0 += kPiece8) {
    const int64_t m = n / 8 - t0 < kPiece8 ? n / 8 - t0 : kPiece8;
    const dim3 grid((unsigned)cdiv(m, 256)), block(256);
    const void *xp = (const char *)x + t0 * 8 * (x_bf16 ? 2 : 4);
    uint8_t *q = codes + 8 * t0, *e = scale + t0 / 4;
    if (fmt == CK_MXINT8) {
      if (x_bf16) hipLaunchKernelGGL((k_ckpt8_quant<CK_MXINT8, true>), grid, block, 0, s, xp, m, q, e);
      else hipLaunchKernelGGL((k_ckpt8_quant<CK_MXINT8, false>), grid, block, 0, s, xp, m, q, e);
    } else {
      if (x_bf16) hipLaunchKernelGGL((k_ckpt8_quant<CK_MXFP8, true>), grid, block, 0, s, xp, m, q, e);
      else hipLaunchKernelGGL((k_ckpt8_quant<CK_MXFP8, false>), grid, block, 0, s, xp, m, q, e);
    }
  }
  return hipGetLastError();
}

hipError_t launch_ckpt8_dequantize(int fmt, const uint8_t *codes, const uint8_t *scale, int64_t n, void *out,
                                   bool out_bf16, hipStream_t s) {
  for (int64_t t0 = 0; t0 < n / 8; t0 += kPiece8) {
    const int64_t m = n / 8 - t0 < kPiece8 ? n / 8 - t0 : kPiece8;
    const dim3 grid((unsigned)cdiv(m, 256)), block(256);
    void *o = (char *)out + t0 * 8 * (out_bf16 ? 2 : 4);
    const uint8_t *q = codes + 8 * t0, *e = scale + t0 / 4;
    if (fmt == CK_MXINT8) {
      if (out_bf16) hipLaunchKernelGGL((k_ckpt8_dequant<CK_MXINT8, true>), grid, block, 0, s, q, e, m, o);
      else hipLaunchKernelGGL((k_ckpt8_dequant<CK_MXINT8, false>), grid, block, 0, s, q, e, m, o);
    } else {
      if (out_bf16) hipLaunchKernelGGL((k_ckpt8_dequant<CK_MXFP8, true>), grid, block, 0, s, q, e, m, o);
      else hipLaunchKernelGGL((k_ckpt8_dequant<CK_MXFP8, false>), grid, block, 0, s, q, e, m, o);
    }
  }
  return hipGetLastError();
}

template <bool BF>
static void glu_forward_f(const GluArgs &a, dim3 grid, hipStream_t s) {
  if (!a.codes) hipLaunchKernelGGL((k_glu_forward<BF, CK_NONE>), grid, dim3(256), 0, s, a);
  else if (a.fmt == CK_MXINT8) hipLaunchKernelGGL((k_glu_forward<BF, CK_MXINT8>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_glu_forward<BF, CK_MXFP8>), grid, dim3(256), 0, s, a);
}

// Calls of many rows go in pieces of whole rows, for the same reason.
static int64_t glu_rows(int I) {
  const int64_t rows = kPiece8 / (I / 8), most = int64_t(1) << 22;
  return rows < most ? rows : most;
}
static GluArgs glu_piece(const GluArgs &a, int64_t r0) {
  GluArgs p = a;
  const int64_t n = r0 * a.I, n2 = 2 * n, left = a.R - r0, most = glu_rows(a.I);
  p.R = left < most ? left : most;
  p.gu = (const char *)a.gu + n2 * (a.src == SRC_F32 ? 4 : a.src == SRC_BF16 ? 2 : 1);
  if (a.gu_scale) p.gu_scale = a.gu_scale + n2 / 32;
  if (a.codes) p.codes = a.codes + n2, p.scale = a.scale + n2 / 32;
  if (a.h) p.h = a.h + n;
  if (a.dh) p.dh = (const char *)a.dh + n * (a.dh_bf16 ? 2 : 4);
  if (a.row_w) p.row_w = a.row_w + r0;
  if (a.dgu) p.dgu = a.dgu + n2;
  if (a.drow) p.drow = a.drow + r0;
  return p;
}

hipError_t launch_glu_forward(const GluArgs &a, hipStream_t s) {
  for (int64_t r0 = 0; r0 < a.R; r0 += glu_rows(a.I)) {
    const GluArgs p = glu_piece(a, r0);
    const dim3 grid((unsigned)cdiv(p.R * (p.I / 8), 256));
    if (p.src == SRC_BF16) glu_forward_f<true>(p, grid, s);
    else glu_forward_f<false>(p, grid, s);
  }
  return hipGetLastError();
}

template <bool DHBF, int WPR>
static void glu_backward_d(const GluArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(a.R, 4 / WPR)), block(256);
  switch (a.src) {
    case SRC_BF16: hipLaunchKernelGGL((k_glu_backward<SRC_BF16, DHBF, WPR>), grid, block, 0, s, a); break;
    case SRC_F32: hipLaunchKernelGGL((k_glu_backward<SRC_F32, DHBF, WPR>), grid, block, 0, s, a); break;
    case SRC_MXINT8: hipLaunchKernelGGL((k_glu_backward<SRC_MXINT8, DHBF, WPR>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_glu_backward<SRC_MXFP8, DHBF, WPR>), grid, block, 0, s, a); break;
  }
}

hipError_t launch_glu_backward(const GluArgs &a, hipStream_t s) {
  // Four waves a row where a row feeds them, or few rows would leave CUs idle. us, one
  // wave a row against four: I = 2880, 8192 rows 43.7 / 38.6, 64 rows 7.4 / 4.3; I = 1024,
  // 256 rows 4.2 / 3.6, 2048 rows 7.2 / 8.0; I = 768, 16384 rows 23.1 / 27.1. (1536, three
  // rounds of a wave, lies between the measured 1024 and 2880.)
  const bool wide = a.I > 1536 || a.R <= 512;
  for (int64_t r0 = 0; r0 < a.R; r0 += glu_rows(a.I)) {
    const GluArgs p = glu_piece(a, r0);
    if (wide && p.dh_bf16) glu_backward_d<true, 4>(p, s);
    else if (wide) glu_backward_d<false, 4>(p, s);
    else if (p.dh_bf16) glu_backward_d<true, 1>(p, s);
    else glu_backward_d<false, 1>(p, s);
  }
  return hipGetLastError();
}

}  // namespace nf4moe
