// The norms around a block, fused with its gate and residual scale.
//
// Forward, per row of H values, one pass over the data:
//   z  = f * rstd_f * w_post          rstd_f = 1 / sqrt(mean f^2 + eps)   (or z = f)
//   x' = round(x + alpha * phi(gate) * z)
//   y  = x' * rstd_x * w_pre          rstd_x of the stored x'
// Backward, from dx' and dy:
//   g  = dx' + rstd_x (dy w_pre - n_x mean(dy w_pre n_x)),  n_x = x' rstd_x
//   dx = g;  dw_pre = sum_t dy n_x
//   dz = alpha phi g;  dgate = alpha phi' g z (summed to the gate's shape)
//   df = rstd_f (dz w_post - n_f mean(dz w_post n_f));  dw_post = sum_t dz n_f
// Everything is fp32 in registers between the loads and the stores; each output
// is rounded once. Both directions are bound by memory traffic.
//
// A row is held by TPR threads, 8 NC values each, so its reductions are a wave
// sum (TPR = 64) or wave sums joined through LDS. Rows of any width: the last
// 8-element piece may be partial, and pieces need no alignment (H odd, views).
#include "ckpt8.h"
#include "internal.h"
#include "train.h"

namespace nf4moe {

namespace {

// Elements i .. i + 7 of a row of H, zeros past the end.
template <bool BF>
__device__ inline void load_row8(const void *p, int64_t base, int i, int H, float (&v)[8]) {
  if (i + 8 <= H) {
    load_elems8<BF>(p, base + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (i + j < H)
        v[j] = BF ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[base + i + j])
                  : reinterpret_cast<const float *>(p)[base + i + j];
    }
  }
}
template <bool BF>
__device__ inline void store_row8(void *p, int64_t base, int i, int H, const float (&v)[8]) {
  if (i + 8 <= H) {
    store_elems8<BF>(p, base + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < H) {
        if (BF) reinterpret_cast<uint16_t *>(p)[base + i + j] = (uint16_t)f32_to_bf16_rne(v[j]);
        else reinterpret_cast<float *>(p)[base + i + j] = v[j];
      }
  }
}

// The gate's factor phi and its slope. tanh by the library function: 1 - 2 / (1 +
// exp(2 v)) loses the small values, where a tanh gate starts.
__device__ inline float gate_phi(int fn, float v) {
  if (fn == 1) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
  return fn == 2 ? tanhf(v) : v;
}
__device__ inline float gate_slope(int fn, float phi) { return fn == 1 ? phi * (1.0f - phi) : fn == 2 ? 1.0f - phi * phi : 1.0f; }

__device__ inline float gate_scalar(const NormArgs &p, int64_t i) {
  return p.gate_bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p.gate)[i]) : reinterpret_cast<const float *>(p.gate)[i];
}
__device__ inline void gate_row8(const NormArgs &p, int64_t base, int i, float (&v)[8]) {
  if (p.gate_bf16) load_row8<true>(p.gate, base, i, p.H, v);
  else load_row8<false>(p.gate, base, i, p.H, v);
}

// Sum over the TPR threads of a row (NV values at once); red has a place per
// wave and value. TPR > 64: two barriers, taken by every thread of the workgroup.
template <int TPR, int NV>
__device__ inline void row_sum(float (&v)[NV], float *red) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = wave_sum(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < NV; ++k) red[wave * NV + k] = v[k];
    }
    lds_barrier();
    const int first = (int)(threadIdx.x / TPR) * W;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[(first + w) * NV + k];
      v[k] = s;
    }
    lds_barrier();  // red may be written again
  }
}

template <bool XBF, int TPR, int NC>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm_forward(NormArgs p) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  __shared__ float red[THREADS / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  // Rows past the end (TPR = 64 only: no barriers there) leave; else ROWS = 1 or
  // all threads of the workgroup stay for the barriers.
  const bool live = row < p.T;
  const int64_t base = (live ? row : 0) * p.H;
  const int H = p.H;
  float x[NC][8], f[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = 8 * (t + c * TPR);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[c][j] = f[c][j] = 0.0f;
    if (i < H) {
      load_row8<XBF>(p.x, base, i, H, x[c]);
      if (p.f) load_row8<true>(p.f, base, i, H, f[c]);
    }
  }
  if (p.f) {
    float rs = 1.0f;
    if (p.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] += f[c][j] * f[c][j];
      row_sum<TPR, 1>(ss, red);
      rs = 1.0f / sqrtf(ss[0] / (float)H + p.eps);
      if (t == 0 && live) p.rstd_post[row] = rs;
    }
    const float row_gate = p.gate_kind == 2 ? gate_phi(p.gate_fn, gate_scalar(p, live ? row : 0)) : 1.0f;
    const float m = p.alpha * row_gate;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i < H) {
        float w[8], g[8];
        if (p.w_post) load_row8<false>(p.w_post, 0, i, H, w);
        if (p.gate_kind & 1) gate_row8(p, p.gate_kind == 3 ? base : 0, i, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = p.w_post ? f[c][j] * rs * w[j] : f[c][j];
          const float k = (p.gate_kind & 1) ? m * gate_phi(p.gate_fn, g[j]) : m;
          x[c][j] += k * z;
          if (XBF) x[c][j] = bf16_to_f32(f32_to_bf16_rne(x[c][j]));
        }
        if (live) store_row8<XBF>(p.x_new, base, i, H, x[c]);
      }
    }
  }
  if (p.w_pre) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += x[c][j] * x[c][j];
    row_sum<TPR, 1>(ss, red);
    const float rs = 1.0f / sqrtf(ss[0] / (float)H + p.eps);
    if (t == 0 && live) p.rstd_pre[row] = rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i < H) {
        float w[8], y[8];
        load_row8<false>(p.w_pre, 0, i, H, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[c][j] * rs * w[j];
        if (live) store_row8<true>(p.y, base, i, H, y);
      }
    }
  }
}

// Rows are dealt to a fixed number of workgroups (a function of T and H), each
// row slot of a workgroup keeps its columns' sums for dw_pre, dw_post and a
// per-channel dgate in registers, the slots are added in order through LDS, and
// k_norm_colsum adds the workgroups in order: the same bits on every run.
template <bool XBF, int TPR, int NC>
__global__ __launch_bounds__(1024) void k_norm_backward(NormArgs p) {
  constexpr int SLOTS = 1024 / TPR;
  __shared__ float red[2 * 16];
  extern __shared__ float slot_sum[];  // [3][H] (SLOTS > 1: at most 48 KB)
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int H = p.H;
  float a_pre[NC][8] = {}, a_post[NC][8] = {}, a_gate[NC][8] = {};
  const float invH = 1.0f / (float)H;
  // every thread runs the same number of rounds: row_sum's barriers need them all
  for (int64_t r0 = (int64_t)blockIdx.x * SLOTS; r0 < p.T; r0 += (int64_t)gridDim.x * SLOTS) {
    const int64_t row = r0 + slot;
    const bool live = row < p.T;
    const int64_t base = (live ? row : 0) * H;
    float g[NC][8], f[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[c][j] = f[c][j] = 0.0f;
      if (i < H && live) {
        if (p.dx_new) load_row8<XBF>(p.dx_new, base, i, H, g[c]);
        if (p.f) load_row8<true>(p.f, base, i, H, f[c]);
      }
    }
    if (p.w_pre) {
      float dy[NC][8], n[NC][8];
      float s[1] = {0.0f};
      const float rs = live ? p.rstd_pre[row] : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[c][j] = n[c][j] = 0.0f;
        if (i < H && live) {
          float w[8];
          load_row8<true>(p.dy, base, i, H, dy[c]);
          load_row8<XBF>(p.x, base, i, H, n[c]);
          load_row8<false>(p.w_pre, 0, i, H, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            n[c][j] *= rs;
            a_pre[c][j] += dy[c][j] * n[c][j];
            dy[c][j] *= w[j];
            s[0] += dy[c][j] * n[c][j];
          }
        }
      }
      row_sum<TPR, 1>(s, red);
      const float mean = s[0] * invH;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[c][j] += rs * (dy[c][j] - n[c][j] * mean);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i < H && live) store_row8<XBF>(p.dx, base, i, H, g[c]);
    }
    if (p.f) {
      // f becomes n_f (or stays f), g becomes dz * w_post (or dz)
      const float rs = p.w_post ? (live ? p.rstd_post[row] : 0.0f) : 1.0f;
      const float raw = p.gate_kind == 2 ? gate_phi(p.gate_fn, gate_scalar(p, live ? row : 0)) : 1.0f;
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
        if (i < H && live) {
          float w[8], v[8], dg[8];
          if (p.w_post) load_row8<false>(p.w_post, 0, i, H, w);
          if (p.gate_kind & 1) gate_row8(p, p.gate_kind == 3 ? base : 0, i, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float n = f[c][j] * rs, wj = p.w_post ? w[j] : 1.0f;
            const float phi = (p.gate_kind & 1) ? gate_phi(p.gate_fn, v[j]) : raw;
            const float gz = p.alpha * g[c][j] * n * wj;  // alpha g z
            dg[j] = gz * gate_slope(p.gate_fn, phi);
            if (p.gate_kind == 1) a_gate[c][j] += dg[j];
            s[1] += gz;
            const float dz = p.alpha * phi * g[c][j];
            if (p.w_post) a_post[c][j] += dz * n;
            f[c][j] = n;
            g[c][j] = dz * wj;
            s[0] += g[c][j] * n;
          }
          if (p.gate_kind == 3) store_row8<false>(p.dgate, base, i, H, dg);
        }
      }
      row_sum<TPR, 2>(s, red);
      if (p.gate_kind == 2 && t == 0 && live) p.dgate[row] = s[1] * gate_slope(p.gate_fn, raw);
      const float mean = s[0] * invH;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
        if (i < H && live) {
          if (p.w_post) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[c][j] = rs * (g[c][j] - f[c][j] * mean);
          }
          store_row8<true>(p.df, base, i, H, g[c]);
        }
      }
    }
  }
  // join the slots, then one partial per workgroup
  float *out = p.partial + (int64_t)blockIdx.x * 3 * H;
  for (int s = 0; s < SLOTS; ++s) {
    if (slot == s) {
      float *dst = SLOTS == 1 ? out : slot_sum;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * (t + c * TPR) + j;
          if (i >= H) continue;
          const bool first = s == 0;
          dst[i] = first ? a_pre[c][j] : dst[i] + a_pre[c][j];
          dst[H + i] = first ? a_post[c][j] : dst[H + i] + a_post[c][j];
          dst[2 * H + i] = first ? a_gate[c][j] : dst[2 * H + i] + a_gate[c][j];
        }
      }
    }
    if (SLOTS > 1) lds_barrier();
  }
  if (SLOTS > 1)
    for (int i = threadIdx.x; i < 3 * H; i += 1024) out[i] = slot_sum[i];
}

// dw_pre, dw_post and dgate [H] from the workgroups' partial sums: 64 columns a
// workgroup, 16 waves each adding every 16th partial in order, then the waves in
// order.
__global__ __launch_bounds__(1024) void k_norm_colsum(NormArgs p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane, which = blockIdx.y;
  float *out = which == 0 ? p.dw_pre : which == 1 ? p.dw_post : (p.gate_kind == 1 ? p.dgate : nullptr);
  if (!out) return;  // the whole workgroup
  float s = 0.0f;
  if (col < p.H)
    for (int g = wave; g < p.groups; g += 16) s += p.partial[((int64_t)g * 3 + which) * p.H + col];
  part[wave][lane] = s;
  lds_barrier();
  if (wave != 0 || col >= p.H) return;
  for (int w = 1; w < 16; ++w) s += part[w][lane];
  out[col] = s;
}

template <bool XBF>
hipError_t norm_forward_t(const NormArgs &a, hipStream_t s) {
  if (a.H <= 512)
    hipLaunchKernelGGL((k_norm_forward<XBF, 64, 1>), dim3((unsigned)cdiv(a.T, 4)), dim3(256), 0, s, a);
  else if (a.H <= 2048)
    hipLaunchKernelGGL((k_norm_forward<XBF, 256, 1>), dim3((unsigned)a.T), dim3(256), 0, s, a);
  else if (a.H <= 4096)
    hipLaunchKernelGGL((k_norm_forward<XBF, 512, 1>), dim3((unsigned)a.T), dim3(512), 0, s, a);
  else if (a.H <= 8192)
    hipLaunchKernelGGL((k_norm_forward<XBF, 1024, 1>), dim3((unsigned)a.T), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_forward<XBF, 1024, 2>), dim3((unsigned)a.T), dim3(1024), 0, s, a);
  return hipGetLastError();
}

int norm_slots(int H) { return H <= 512 ? 16 : H <= 2048 ? 4 : H <= 4096 ? 2 : 1; }

template <bool XBF>
hipError_t norm_backward_t(const NormArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)a.groups), block(1024);
  const size_t lds = norm_slots(a.H) > 1 ? (size_t)3 * a.H * sizeof(float) : 0;
  if (a.H <= 512) hipLaunchKernelGGL((k_norm_backward<XBF, 64, 1>), grid, block, lds, s, a);
  else if (a.H <= 2048) hipLaunchKernelGGL((k_norm_backward<XBF, 256, 1>), grid, block, lds, s, a);
  else if (a.H <= 4096) hipLaunchKernelGGL((k_norm_backward<XBF, 512, 1>), grid, block, lds, s, a);
  else if (a.H <= 8192) hipLaunchKernelGGL((k_norm_backward<XBF, 1024, 1>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_norm_backward<XBF, 1024, 2>), grid, block, lds, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dw_pre || a.dw_post || (a.dgate && a.gate_kind == 1)) {
    hipLaunchKernelGGL(k_norm_colsum, dim3((unsigned)cdiv(a.H, 64), 3), dim3(1024), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Workgroups of the backward: one per CU (1024 threads each), fewer where there
// are fewer rows.
int norm_backward_groups(int64_t T, int H) {
  const int64_t need = cdiv(T, norm_slots(H));
  return (int)(need < 256 ? need : 256);
}

hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s) {
  return a.x_bf16 ? norm_forward_t<true>(a, s) : norm_forward_t<false>(a, s);
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s) {
  return a.x_bf16 ? norm_backward_t<true>(a, s) : norm_backward_t<false>(a, s);
}

}  // namespace nf4moe
