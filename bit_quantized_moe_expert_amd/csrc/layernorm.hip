// Layer norm of [T, H] rows, forward and backward.
//
// Forward: y = (x - mean) rstd w + b with rstd = 1 / sqrt(mean((x - mean)^2) + eps). The first sum's mean is
// off by up to (24 + H / 64) 2^-24 of the row's size, more than the spread of a row that lies far from
// zero. The values centred by it are exact there; their own mean dm and that of their squares come from a second exchange
// over registers, and dm is taken out of both: what is left of the error is as small a part of dm again
// (rows of 10000.1, H 2880: y off by 0.53 without this, by less than 10^-6 with it; 0 to 3 % of the time, 6 % of rows of 16384).
// Backward, with n = (x - mean) rstd and a = dy w:
//   dx = dx_base + rstd (a - mean(a) - n mean(a n));  dw = sum_t dy n;  db = sum_t dy
// Everything is fp32 in registers, each output rounded once. Both directions are bound by memory
// traffic. Rows lie as in the block norms' kernels: TPR threads a row, 8 NC values each, so that a row is read
// once and a sum meets in one exchange through LDS. Measured, us: 8190 x 2880 fp32 to bf16 28.5 to 29 (142
// MB, 4.9 to 5.0 TB/s, a copy's rate 5.4); backward of 8192 x 2048 bf16 with a base 27 (134 MB, 5.0 TB/s) and
// 4 for the column sums; 4 rows 3.0.
#include "dense.h"
#include "internal.h"
#include "rows.h"

namespace nf4moe {

namespace {

template <bool XBF, bool YBF, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_ln_forward(LayerNormArgs p) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  __shared__ float red[THREADS / 64], red2[2 * THREADS / 64];
  const int t = threadIdx.x % TPR, H = p.H;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const bool live = row < p.T;   // rows past the end read row 0 and store nothing
  const int64_t base = (live ? row : 0) * H;
  Raw8<XBF> raw[NC] = {};
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (8 * (t + c * TPR) < H) raw[c] = load_raw8<XBF, ODD>(p.x, base, 8 * (t + c * TPR), H);
  float x[NC][8], s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    unpack_raw8<XBF, ODD>(raw[c], 8 * (t + c * TPR), H, x[c]);   // zeros past the row's end
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += x[c][j];
  }
  row_sum<TPR, 1>(s, red);
  const float first = s[0] / (float)H;
  float c2[2] = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[c][j] = 8 * (t + c * TPR) + j < H ? x[c][j] - first : 0.0f;
      c2[0] += x[c][j];
      c2[1] += x[c][j] * x[c][j];
    }
  row_sum<TPR, 2>(c2, red2);
  const float dm = c2[0] / (float)H, v2 = c2[1] / (float)H - dm * dm;
  const float rs = 1.0f / sqrtf((v2 < 0.0f ? 0.0f : v2) + p.eps);   // (a NaN stays one)
  if (!live) return;
  if (t == 0) p.mean[row] = first + dm, p.rstd[row] = rs;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = 8 * (t + c * TPR);
    if (i >= H) continue;
    float y[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (x[c][j] - dm) * rs;
    if (p.w) {
      load_row8<false, ODD>(p.w, 0, i, H, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= v[j];
    }
    if (p.b) {
      load_row8<false, ODD>(p.b, 0, i, H, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] += v[j];
    }
    store_row8<YBF, ODD>(p.y, base, i, H, y);
  }
}

// Rows are dealt to a fixed number of workgroups (a function of T and H); each row slot of a
// workgroup keeps its columns' two sums in registers, the slots are added in order through LDS and
// k_ln_colsum adds the workgroups in order: the same bits on every run.
__host__ __device__ constexpr int back_threads(int tpr) { return tpr <= 512 ? 512 : 1024; }

template <bool XBF, bool YBF, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(back_threads(TPR)) void k_ln_backward(LayerNormArgs p) {
  constexpr int THREADS = back_threads(TPR), SLOTS = THREADS / TPR;
  __shared__ float red[2][2 * THREADS / 64];   // in turn for even and odd rounds
  extern __shared__ float slot_sum[];          // [2][H] (SLOTS > 1, H <= 2048: at most 16 KB)
  const int t = threadIdx.x % TPR, H = p.H;
  const int slot = TPR >= 64 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR) : (int)threadIdx.x / TPR;
  const float invH = 1.0f / (float)H;
  float w[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) w[c][j] = 1.0f;
  if (p.w) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (8 * (t + c * TPR) < H) load_row8<false, ODD>(p.w, 0, 8 * (t + c * TPR), H, w[c]);
  }
  float sw[NC][8] = {}, sb[NC][8] = {};
  int turn = 0;
  // every thread runs the same number of rounds: row_sum's barriers need them all
  for (int64_t r0 = (int64_t)blockIdx.x * SLOTS; r0 < p.T; r0 += (int64_t)gridDim.x * SLOTS) {
    const int64_t row = r0 + slot;
    const bool live = row < p.T;
    const int64_t base = (live ? row : 0) * H;
    turn ^= 1;
    Raw8<XBF> rx[NC] = {}, rb[NC] = {};
    Raw8<YBF> ry[NC] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i >= H || !live) continue;
      ry[c] = load_raw8<YBF, ODD>(p.dy, base, i, H);
      rx[c] = load_raw8<XBF, ODD>(p.x, base, i, H);
      if (p.dx_base && p.dx) rb[c] = load_raw8<XBF, ODD>(p.dx_base, base, i, H);
    }
    const float mean = live ? p.mean[row] : 0.0f, rs = live ? p.rstd[row] : 0.0f;
    float a[NC][8], n[NC][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      unpack_raw8<YBF, ODD>(ry[c], i, H, a[c]);
      unpack_raw8<XBF, ODD>(rx[c], i, H, n[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // past the row's end dy is zero and so are all its products but those with a NaN mean
        n[c][j] = i + j < H && live ? (n[c][j] - mean) * rs : 0.0f;
        sb[c][j] += a[c][j];
        sw[c][j] += a[c][j] * n[c][j];
        a[c][j] *= w[c][j];
        s[0] += a[c][j];
        s[1] += a[c][j] * n[c][j];
      }
    }
    if (!p.dx) continue;   // the whole grid
    row_sum<TPR, 2>(s, red[turn]);
    if (!live) continue;
    const float ma = s[0] * invH, mn = s[1] * invH;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i >= H) continue;
      float d[8];
      unpack_raw8<XBF, ODD>(rb[c], i, H, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] += rs * (a[c][j] - ma - n[c][j] * mn);
      store_row8<XBF, ODD>(p.dx, base, i, H, d);
    }
  }
  if (!p.dw && !p.db) return;   // the whole grid
  float *out = p.partial + (int64_t)blockIdx.x * 2 * H;
  // the slots of a wave by exchanges, then the waves (or wider slots) in order
  constexpr int IN_WAVE = TPR < 64 ? 64 / TPR : 1;
  if constexpr (IN_WAVE > 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int d = TPR; d < 64; d *= 2) sw[c][j] += __shfl_xor(sw[c][j], d, kWave), sb[c][j] += __shfl_xor(sb[c][j], d, kWave);
  }
  for (int s = 0; s < SLOTS; s += IN_WAVE) {
    if (slot == s) {
      float *dst = SLOTS == 1 ? out : slot_sum;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * (t + c * TPR) + j;
          if (i >= H) continue;
          dst[i] = s == 0 ? sw[c][j] : dst[i] + sw[c][j];
          dst[H + i] = s == 0 ? sb[c][j] : dst[H + i] + sb[c][j];
        }
    }
    if (SLOTS > 1) lds_barrier();
  }
  if (SLOTS > 1)
    for (int i = threadIdx.x; i < 2 * H; i += THREADS) out[i] = slot_sum[i];
}

// dw and db from the workgroups' partial sums: 64 columns a workgroup, 16 waves each adding
// every 16th partial in order, then the waves in order.
__global__ __launch_bounds__(1024) void k_ln_colsum(LayerNormArgs p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane, which = blockIdx.y;
  float *out = which == 0 ? p.dw : p.db;
  if (!out) return;   // the whole workgroup
  float s = 0.0f;
  if (col < p.H) {
#pragma unroll 8
    for (int g = wave; g < p.groups; g += 16) s += p.partial[((int64_t)g * 2 + which) * p.H + col];
  }
  part[wave][lane] = s;
  lds_barrier();
  if (wave != 0 || col >= p.H) return;
  for (int w = 1; w < 16; ++w) s += part[w][lane];
  out[col] = s;
}

// Backward: the fewest threads that a row fits, 8 values each (2^20 rows of 64 by 64 threads each: 289 us, by 8
// 71; more values a thread cost registers, whose sums they hold).
int ln_tpr(int H) {
  int n = 8;
  while (n < 1024 && 8 * n < H) n *= 2;
  return n;
}
int ln_slots(int H) { return back_threads(ln_tpr(H)) / ln_tpr(H); }

// f(TPR, NC) as integral constants, by the width of a row.
template <class F>
void by_width(int H, F &&f) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  switch (ln_tpr(H)) {
    case 8: return f(integral_constant<int, 8>(), one);
    case 16: return f(integral_constant<int, 16>(), one);
    case 32: return f(integral_constant<int, 32>(), one);
    case 64: return f(integral_constant<int, 64>(), one);
    case 128: return f(integral_constant<int, 128>(), one);
    case 256: return f(integral_constant<int, 256>(), one);
    case 512: return f(integral_constant<int, 512>(), one);
    default:
      if (H <= 8192) return f(integral_constant<int, 1024>(), one);
      return f(integral_constant<int, 1024>(), integral_constant<int, 2>());
  }
}
// Forward: up to 32 values a thread, whose loads go out together, and so fewer waves to a row's sum (8190 x
// 2880 bf16: 512 threads of 8 values 24.6 us, 128 of 24 19.5; 4096 x 4096 fp32 22.0 and 19.0); 16 above 4096, where
// many rows ran slower with 32 (16384 x 8192 bf16: 8 values 138, 16 121, 32 140). A few rows, whose time is one
// row's, take 8 (4 x 2048: 3.0 and 4.0).
template <class F>
void by_width_forward(int64_t T, int H, F &&f) {
  using std::integral_constant;
  if (T <= 256 || H <= 512) return by_width(H, f);
  const auto more = [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    if (H <= 24 * TPR) f(tpr, integral_constant<int, 3>());
    else f(tpr, integral_constant<int, 4>());
  };
  const integral_constant<int, 64> wave;
  if (H <= 1024) f(wave, integral_constant<int, 2>());
  else if (H <= 2048) more(wave);
  else if (H <= 4096) more(integral_constant<int, 128>());
  else if (H <= 8192) f(integral_constant<int, 512>(), integral_constant<int, 2>());
  else f(integral_constant<int, 1024>(), integral_constant<int, 2>());
}
// f(XBF, YBF, ODD)
template <class F>
void by_types(const LayerNormArgs &a, F &&f) {
  const bool odd = a.H % 8 != 0;
  std::true_type y;
  std::false_type n;
  if (a.x_bf16 && a.y_bf16) odd ? f(y, y, y) : f(y, y, n);
  else if (a.x_bf16) odd ? f(y, n, y) : f(y, n, n);
  else if (a.y_bf16) odd ? f(n, y, y) : f(n, y, n);
  else odd ? f(n, n, y) : f(n, n, n);
}

}  // namespace

int layer_norm_groups(int64_t T, int H) {
  const int64_t need = cdiv(T, ln_slots(H)), most = 256 * 1024 / back_threads(ln_tpr(H));
  return (int)(need < most ? need : most);
}

// Many rows go in pieces, each well inside a dispatch's 2^32 threads.
hipError_t launch_layer_norm_forward(const LayerNormArgs &a, hipStream_t s) {
  constexpr int64_t kPiece = 1 << 21;
  for (int64_t r0 = 0; r0 < a.T; r0 += kPiece) {
    LayerNormArgs p = a;
    const int64_t n = r0 * a.H;
    p.T = a.T - r0 < kPiece ? a.T - r0 : kPiece;
    p.x = (const char *)a.x + n * (a.x_bf16 ? 2 : 4), p.y = (char *)a.y + n * (a.y_bf16 ? 2 : 4);
    p.mean = a.mean + r0, p.rstd = a.rstd + r0;
    by_types(p, [&](auto xb, auto yb, auto odd) {
      by_width_forward(a.T, p.H, [&](auto tpr, auto nc) {
        constexpr int threads = tpr.value > 256 ? tpr.value : 256;
        hipLaunchKernelGGL((k_ln_forward<xb.value, yb.value, tpr.value, nc.value, odd.value>),
                           dim3((unsigned)cdiv(p.T, threads / tpr.value)), dim3(threads), 0, s, p);
      });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_layer_norm_backward(const LayerNormArgs &a, hipStream_t s) {
  const size_t lds = ln_slots(a.H) > 1 ? (size_t)2 * a.H * sizeof(float) : 0;
  by_types(a, [&](auto xb, auto yb, auto odd) {
    by_width(a.H, [&](auto tpr, auto nc) {
      hipLaunchKernelGGL((k_ln_backward<xb.value, yb.value, tpr.value, nc.value, odd.value>), dim3((unsigned)a.groups),
                         dim3(back_threads(tpr.value)), lds, s, a);
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dw && !a.db)) return e;
  hipLaunchKernelGGL(k_ln_colsum, dim3((unsigned)cdiv(a.H, 64), 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4moe
