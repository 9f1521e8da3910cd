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
// is rounded once. Both directions are bound by memory traffic: the forward of 8190 x
// 2880 (fp32 stream, 283 MB) takes 52.4 us, 5.4 TB/s, the backward of 8192 x 2048 bf16
// (201 MB) 43.4 us and 5.0 for the joined column sums, 4.2 TB/s: a row's two sums wait
// for each other. Wider rows, bf16: 4096 x 4096 25.7 and 54.3 us, 4096 x 8192 51.5 and
// 95.8, 2048 x 16384 50.9 and 119.8. Above 8192 columns a thread of the backward holds two
// pieces, and its registers do not suffice: 8 to 92 of them go to memory (36 to 304 bytes a
// lane, most where H % 8 != 0; 2048 x 16383 fp32 with a gate per element 319 us).
//
// A row is held by TPR threads, 8 NC values each, so its reductions are a wave
// sum (TPR = 64) or wave sums joined through LDS. Rows of any width: the last
// 8-element piece may be partial, and pieces need no alignment (H odd, views).
#include "ckpt8.h"
#include "internal.h"
#include "train.h"

namespace nf4moe {

namespace {

// Eight elements as they lie in memory: loads first, arithmetic later. ODD: H % 8 != 0,
// a row's last piece is partial; then its lane reads the row's last eight elements, which
// are all there, and unpack_raw8 moves its own ones down and zeros in behind them. One
// load for every lane, no branch between loads, nothing read past the row; a load per
// element in that lane made the kernels twice as long (7954 rows of 118 bf16, backward:
// 23 us against 13.5 for 120 columns).
template <bool BF>
struct Raw8 {
  uint4 v[BF ? 1 : 2];
};
template <bool BF, bool ODD>
__device__ inline Raw8<BF> load_raw8(const void *p, int64_t base, int i, int H) {
  Raw8<BF> r;
  if (!ODD || H >= 8) {
    const char *at = reinterpret_cast<const char *>(p) + (base + (ODD ? min(i, H - 8) : i)) * (BF ? 2 : 4);
    r.v[0] = load16(at);
    if constexpr (!BF) r.v[1] = load16(at + 16);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = base + min(j, H - 1);  // (i is 0)
      w[j] = BF ? (uint32_t)reinterpret_cast<const uint16_t *>(p)[at] : reinterpret_cast<const uint32_t *>(p)[at];
      w[j] = j < H ? w[j] : 0u;
    }
    if constexpr (BF) {
      r.v[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    } else {
      r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
      r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  return r;
}
template <int N>
__device__ inline void move_down(uint32_t (&w)[N], int by, bool yes) {
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = yes ? (k + by < N ? w[k + by] : 0u) : w[k];
}
template <bool BF, bool ODD>
__device__ inline void unpack_raw8(const Raw8<BF> &r, int i, int H, float (&v)[8]) {
  const int down = ODD && H >= 8 ? max(i - (H - 8), 0) : 0;  // places that the piece began too early
  if constexpr (BF) {
    uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
    if constexpr (ODD) {
      move_down(w, 2, down & 4);
      move_down(w, 1, down & 2);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = down & 1 ? __builtin_amdgcn_alignbit(k < 3 ? w[k + 1] : 0u, w[k], 16) : w[k];
    }
    unpack_bf16x8(make_uint4(w[0], w[1], w[2], w[3]), v);
  } else {
    uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
    if constexpr (ODD) {
      move_down(w, 4, down & 4);
      move_down(w, 2, down & 2);
      move_down(w, 1, down & 1);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  }
}
// Elements i .. i + 7 of a row of H (i < H), zeros past the end, and back.
template <bool BF, bool ODD>
__device__ inline void load_row8(const void *p, int64_t base, int i, int H, float (&v)[8]) {
  unpack_raw8<BF, ODD>(load_raw8<BF, ODD>(p, base, i, H), i, H, v);
}
template <bool BF, bool ODD>
__device__ inline void store_row8(void *p, int64_t base, int i, int H, const float (&v)[8]) {
  if (!ODD || i + 8 <= H) {
    store_elems8<BF>(p, base + i, v);
    return;
  }
  // the partial piece: 4 elements, then 2, then 1, those that its length has
  const int n = H & 7;
  const uint32_t four = n & 4 ? ~0u : 0u, two = n & 2 ? ~0u : 0u;
  auto pick = [](uint32_t m, uint32_t a, uint32_t b) { return (m & a) | (~m & b); };
  if constexpr (BF) {
    uint16_t *at = reinterpret_cast<uint16_t *>(p) + base + i;
    const uint4 w = pack_bf16x8(v);
    if (n & 4) store8(at, make_uint2(w.x, w.y));
    if (n & 2) store4(at + (n & 4), pick(four, w.z, w.x));
    if (n & 1) at[n & 6] = (uint16_t)pick(two, pick(four, w.w, w.y), pick(four, w.z, w.x));
  } else {
    uint32_t *at = reinterpret_cast<uint32_t *>(p) + base + i;
    uint32_t w[7];
#pragma unroll
    for (int k = 0; k < 7; ++k) w[k] = __float_as_uint(v[k]);
    if (n & 4) store16(at, make_uint4(w[0], w[1], w[2], w[3]));
    if (n & 2) store8(at + (n & 4), make_uint2(pick(four, w[4], w[0]), pick(four, w[5], w[1])));
    if (n & 1) at[n & 6] = pick(two, pick(four, w[6], w[2]), pick(four, w[4], w[0]));
  }
}

// The gate's factor phi and its slope at gate value v. tanh by the library function: 1 - 2 /
// (1 + exp(2 v)) loses the small values, where a tanh gate starts. The slopes from v, not from
// phi: where the gate saturates, 1 - phi (1 - phi^2) has lost its bits (sigma's was 0 from v = 17,
// tanh's from |v| = 9 and 6 % off at 8). With e = exp(-|v|) (exp(-2 |v|)) they are e / (1 + e)^2
// (four times that), which lose none.
__device__ inline float gate_phi(int fn, float v) {
  if (fn == 1) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
  return fn == 2 ? tanhf(v) : v;
}
__device__ inline float gate_slope(int fn, float v) {
  if (fn == 0) return 1.0f;
  const float e = __builtin_amdgcn_exp2f(fabsf(v) * (fn == 1 ? -1.44269504088896341f : -2.88539008177792681f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return (fn == 1 ? e : 4.0f * e) * r * r;
}

// phi of 8 gate values; the function is chosen once, outside the loop over them.
__device__ inline void gate_phi8(int fn, const float (&v)[8], float (&phi)[8]) {
  if (fn == 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) phi[j] = gate_phi(1, v[j]);
  } else if (fn == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) phi[j] = gate_phi(2, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) phi[j] = v[j];
  }
}

__device__ inline float gate_scalar(const NormArgs &p, int64_t i) {
  return p.gate_bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p.gate)[i]) : reinterpret_cast<const float *>(p.gate)[i];
}
template <bool ODD>
__device__ inline void gate_row8(const NormArgs &p, int64_t base, int i, float (&v)[8]) {
  if (p.gate_bf16) load_row8<true, ODD>(p.gate, base, i, p.H, v);
  else load_row8<false, ODD>(p.gate, base, i, p.H, v);
}

// Sum over the TPR threads of a row (NV values at once); red has a place per wave and
// value. TPR > 64: one barrier, taken by every thread of the workgroup. Consecutive
// sums use different places (a thread that writes them again has passed another
// sum's barrier, and so has every reader).
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
  }
}

template <bool XBF, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm_forward(NormArgs p) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  __shared__ float red[2][THREADS / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  // Rows past the end (TPR = 64) read row 0 and store nothing.
  const bool live = row < p.T;
  const int64_t base = (live ? row : 0) * p.H;
  const int H = p.H;
  Raw8<XBF> rx[NC] = {};
  Raw8<true> rf[NC] = {};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = 8 * (t + c * TPR);
    if (i >= H) continue;
    rx[c] = load_raw8<XBF, ODD>(p.x, base, i, H);
    if (p.f) rf[c] = load_raw8<true, ODD>(p.f, base, i, H);
  }
  float x[NC][8], f[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    unpack_raw8<XBF, ODD>(rx[c], 8 * (t + c * TPR), H, x[c]);
    unpack_raw8<true, ODD>(rf[c], 8 * (t + c * TPR), H, f[c]);
  }
  if (p.f) {
    float rs = 1.0f;
    if (p.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] += f[c][j] * f[c][j];
      row_sum<TPR, 1>(ss, red[0]);
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
        if (p.w_post) load_row8<false, ODD>(p.w_post, 0, i, H, w);
        if (p.w_post) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[c][j] *= rs * w[j];
        }
        if (p.gate_kind & 1) {
          gate_row8<ODD>(p, p.gate_kind == 3 ? base : 0, i, g);
          gate_phi8(p.gate_fn, g, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[c][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[c][j] += m * f[c][j];
          if (XBF) x[c][j] = bf16_to_f32(f32_to_bf16_rne(x[c][j]));
        }
        if (live) store_row8<XBF, ODD>(p.x_new, base, i, H, x[c]);
      }
    }
  }
  if (p.w_pre) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += x[c][j] * x[c][j];
    row_sum<TPR, 1>(ss, red[1]);
    const float rs = 1.0f / sqrtf(ss[0] / (float)H + p.eps);
    if (t == 0 && live) p.rstd_pre[row] = rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i < H) {
        float w[8], y[8];
        load_row8<false, ODD>(p.w_pre, 0, i, H, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[c][j] * rs * w[j];
        if (live) store_row8<true, ODD>(p.y, base, i, H, y);
      }
    }
  }
}

// Rows are dealt to a fixed number of workgroups (a function of T and H). Each row
// slot of a workgroup keeps two sums per column in registers: dy n_x for dw_pre, and
// the one that dw_post and a per-channel dgate both are multiples of, sum_t g n_f
// (without the gate's factor where that is a channel's constant). The slots are added
// in order through LDS and k_norm_colsum adds the workgroups in order: the same bits
// on every run.
// Two workgroups of 512 threads a CU where a row's threads fit (8192 x 2048 bf16: 48
// us; one of 1024: 49; one of 768 that asks for the next row early: 51; four of 256:
// 57, whose partial sums cost most).
__host__ __device__ constexpr int back_threads(int tpr) { return tpr <= 512 ? 512 : 1024; }

template <bool XBF, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(back_threads(TPR)) void k_norm_backward(NormArgs p) {
  constexpr int THREADS = back_threads(TPR), SLOTS = THREADS / TPR;
  // the first sum's places and the second's, in turn for even and odd rounds (a
  // round may have one sum only)
  __shared__ float red[2][2 * 16];
  int turn = 0;
  extern __shared__ float slot_sum[];  // [2][H] (SLOTS > 1, H <= 2048: at most 16 KB)
  const int t = threadIdx.x % TPR, slot = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const int H = p.H;
  const float invH = 1.0f / (float)H;
  // w_pre, and w_post times a per-channel gate's phi, are kept in LDS as each thread
  // reads them (NC = 1)
  constexpr bool KEEP = NC == 1;
  __shared__ float4 kept[KEEP ? 2 : 1][2][KEEP ? TPR : 1];
  auto first_weights = [&](int i, float (&w)[8]) { load_row8<false, ODD>(p.w_pre, 0, i, H, w); };
  auto second_weights = [&](int i, float (&w)[8]) {
    if (p.w_post) {
      load_row8<false, ODD>(p.w_post, 0, i, H, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    }
    if (p.gate_kind == 1) {
      float v[8], phi[8];
      gate_row8<ODD>(p, 0, i, v);
      gate_phi8(p.gate_fn, v, phi);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= phi[j];
    }
  };
  auto keep = [&](int which, const float (&w)[8]) {
    kept[which][0][t] = make_float4(w[0], w[1], w[2], w[3]);
    kept[which][1][t] = make_float4(w[4], w[5], w[6], w[7]);
  };
  auto kept8 = [&](int which, float (&w)[8]) {
    const float4 a = kept[which][0][t], b = kept[which][1][t];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  };
  if (KEEP) {
    if (slot == 0 && 8 * t < H) {
      float w[8];
      if (p.w_pre) {
        first_weights(8 * t, w);
        keep(0, w);
      }
      if (p.f) {
        second_weights(8 * t, w);
        keep(1, w);
      }
    }
    lds_barrier();
  }
  float a_pre[NC][8] = {}, a_post[NC][8] = {};
  // every thread runs the same number of rounds: row_sum's barriers need them all
  for (int64_t r0 = (int64_t)blockIdx.x * SLOTS; r0 < p.T; r0 += (int64_t)gridDim.x * SLOTS) {
    const int64_t row = r0 + slot;
    const bool live = row < p.T;
    const int64_t base = (live ? row : 0) * H;
    turn ^= 1;
    // all that the row reads is asked for together
    Raw8<XBF> rg[NC] = {}, rx[NC] = {};
    Raw8<true> rf[NC] = {}, ry[NC] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i >= H || !live) continue;
      if (p.w_pre) {
        ry[c] = load_raw8<true, ODD>(p.dy, base, i, H);
        rx[c] = load_raw8<XBF, ODD>(p.x, base, i, H);
      }
      if (p.dx_new) rg[c] = load_raw8<XBF, ODD>(p.dx_new, base, i, H);
      if (p.f) rf[c] = load_raw8<true, ODD>(p.f, base, i, H);
    }
    float g[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) unpack_raw8<XBF, ODD>(rg[c], 8 * (t + c * TPR), H, g[c]);
    if (p.w_pre) {
      float a[NC][8], n[NC][8];
      float s[1] = {0.0f};
      const float rs = live ? p.rstd_pre[row] : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
        unpack_raw8<true, ODD>(ry[c], i, H, a[c]);
        unpack_raw8<XBF, ODD>(rx[c], i, H, n[c]);
        if (i < H) {
          float w[8];
          if (KEEP) kept8(0, w);
          else first_weights(i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            n[c][j] *= rs;
            a_pre[c][j] += a[c][j] * n[c][j];
            a[c][j] *= w[j];
            s[0] += a[c][j] * n[c][j];
          }
        }
      }
      row_sum<TPR, 1>(s, red[turn]);
      const float mean = s[0] * invH;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[c][j] += rs * (a[c][j] - n[c][j] * mean);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = 8 * (t + c * TPR);
      if (i < H && live) store_row8<XBF, ODD>(p.dx, base, i, H, g[c]);
    }
    if (p.f) {
      // f becomes n_f (or stays f), g becomes the gradient of n_f up to the factor m
      const float rs = p.w_post ? (live ? p.rstd_post[row] : 0.0f) : 1.0f;
      const float rg = p.gate_kind == 2 ? gate_scalar(p, live ? row : 0) : 0.0f;
      const float phi = p.gate_kind == 2 ? gate_phi(p.gate_fn, rg) : 1.0f;
      const float m = p.alpha * phi;
      float f[NC][8];
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
        unpack_raw8<true, ODD>(rf[c], i, H, f[c]);
        if (i < H) {
          float w[8];
          if (KEEP) kept8(1, w);
          else second_weights(i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[c][j] *= rs;
          if (p.gate_kind == 3) {
            float q[8], dg[8];
            gate_row8<ODD>(p, base, i, q);
#pragma unroll
            for (int j = 0; j < 8; ++j) dg[j] = p.alpha * gate_slope(p.gate_fn, q[j]) * g[c][j] * f[c][j] * w[j];
            gate_phi8(p.gate_fn, q, q);
            if (live) store_row8<false, ODD>(p.dgate, base, i, H, dg);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[c][j] *= q[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) a_post[c][j] += (p.gate_kind == 2 ? phi * g[c][j] : g[c][j]) * f[c][j];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            g[c][j] *= w[j];
            s[0] += g[c][j] * f[c][j];
          }
        }
      }
      row_sum<TPR, 1>(s, red[turn] + 16);
      if (p.gate_kind == 2 && t == 0 && live) p.dgate[row] = p.alpha * s[0] * gate_slope(p.gate_fn, rg);
      const float mean = p.w_post ? s[0] * invH : 0.0f, mr = m * rs;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = 8 * (t + c * TPR);
        if (i < H && live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[c][j] = mr * (g[c][j] - f[c][j] * mean);
          store_row8<true, ODD>(p.df, base, i, H, g[c]);
        }
      }
    }
  }
  // join the slots, then one partial per workgroup
  float *out = p.partial + (int64_t)blockIdx.x * 2 * H;
  for (int s = 0; s < SLOTS; ++s) {
    if (slot == s) {
      float *dst = SLOTS == 1 ? out : slot_sum;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * (t + c * TPR) + j;
          if (i >= H) continue;
          dst[i] = s == 0 ? a_pre[c][j] : dst[i] + a_pre[c][j];
          dst[H + i] = s == 0 ? a_post[c][j] : dst[H + i] + a_post[c][j];
        }
      }
    }
    if (SLOTS > 1) lds_barrier();
  }
  if (SLOTS > 1)
    for (int i = threadIdx.x; i < 2 * H; i += THREADS) out[i] = slot_sum[i];
}

// dw_pre, dw_post and dgate [H] from the workgroups' partial sums: 64 columns a
// workgroup, 16 waves each adding every 16th partial in order, then the waves in
// order.
__global__ __launch_bounds__(1024) void k_norm_colsum(NormArgs p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane, which = blockIdx.y;
  if (which == 0 ? !p.dw_pre : !(p.dw_post || p.gate_kind == 1)) return;  // the whole workgroup
  float s = 0.0f;
  if (col < p.H) {
#pragma unroll 8
    for (int g = wave; g < p.groups; g += 16) s += p.partial[((int64_t)g * 2 + which) * p.H + col];
  }
  part[wave][lane] = s;
  lds_barrier();
  if (wave != 0 || col >= p.H) return;
  for (int w = 1; w < 16; ++w) s += part[w][lane];
  if (which == 0) {
    p.dw_pre[col] = s;
    return;
  }
  s *= p.alpha;
  float phi = 1.0f;
  if (p.gate_kind == 1) {
    const float v = gate_scalar(p, col);
    phi = gate_phi(p.gate_fn, v);
    p.dgate[col] = gate_slope(p.gate_fn, v) * (p.w_post ? p.w_post[col] * s : s);
  }
  if (p.dw_post) p.dw_post[col] = phi * s;
}

template <bool XBF, bool ODD>
hipError_t norm_forward_t(const NormArgs &a, hipStream_t s) {
  if (a.H <= 512)
    hipLaunchKernelGGL((k_norm_forward<XBF, 64, 1, ODD>), dim3((unsigned)cdiv(a.T, 4)), dim3(256), 0, s, a);
  else if (a.H <= 2048)
    hipLaunchKernelGGL((k_norm_forward<XBF, 256, 1, ODD>), dim3((unsigned)a.T), dim3(256), 0, s, a);
  else if (a.H <= 4096)
    hipLaunchKernelGGL((k_norm_forward<XBF, 512, 1, ODD>), dim3((unsigned)a.T), dim3(512), 0, s, a);
  else if (a.H <= 8192)
    hipLaunchKernelGGL((k_norm_forward<XBF, 1024, 1, ODD>), dim3((unsigned)a.T), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_forward<XBF, 1024, 2, ODD>), dim3((unsigned)a.T), dim3(1024), 0, s, a);
  return hipGetLastError();
}

int norm_tpr(int H) { return H <= 512 ? 64 : H <= 2048 ? 256 : H <= 4096 ? 512 : 1024; }
int norm_slots(int H) { return back_threads(norm_tpr(H)) / norm_tpr(H); }

template <bool XBF, bool ODD>
hipError_t norm_backward_t(const NormArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)a.groups), block(back_threads(norm_tpr(a.H)));
  const size_t lds = norm_slots(a.H) > 1 ? (size_t)2 * a.H * sizeof(float) : 0;
  if (a.H <= 512) hipLaunchKernelGGL((k_norm_backward<XBF, 64, 1, ODD>), grid, block, lds, s, a);
  else if (a.H <= 2048) hipLaunchKernelGGL((k_norm_backward<XBF, 256, 1, ODD>), grid, block, lds, s, a);
  else if (a.H <= 4096) hipLaunchKernelGGL((k_norm_backward<XBF, 512, 1, ODD>), grid, block, lds, s, a);
  else if (a.H <= 8192) hipLaunchKernelGGL((k_norm_backward<XBF, 1024, 1, ODD>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_norm_backward<XBF, 1024, 2, ODD>), grid, block, lds, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dw_pre || a.dw_post || (a.dgate && a.gate_kind == 1)) {
    hipLaunchKernelGGL(k_norm_colsum, dim3((unsigned)cdiv(a.H, 64), 2), dim3(1024), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Workgroups of the backward: 1024 threads a CU, fewer where there are fewer rows.
int norm_backward_groups(int64_t T, int H) {
  const int64_t need = cdiv(T, norm_slots(H)), most = 256 * 1024 / back_threads(norm_tpr(H));
  return (int)(need < most ? need : most);
}

// Many rows go in pieces, each well inside a dispatch's 2^32 threads.
hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s) {
  constexpr int64_t kPiece = 1 << 21;
  for (int64_t r0 = 0; r0 < a.T; r0 += kPiece) {
    NormArgs p = a;
    const int64_t n = r0 * a.H, xb = a.x_bf16 ? 2 : 4, gb = a.gate_bf16 ? 2 : 4;
    p.T = a.T - r0 < kPiece ? a.T - r0 : kPiece;
    p.x = (const char *)a.x + n * xb;
    if (a.f) p.f = a.f + n, p.x_new = (char *)a.x_new + n * xb;
    if (a.y) p.y = a.y + n;
    if (a.gate_kind >= 2) p.gate = (const char *)a.gate + (a.gate_kind == 3 ? n : r0) * gb;
    if (a.rstd_post) p.rstd_post = a.rstd_post + r0;
    if (a.rstd_pre) p.rstd_pre = a.rstd_pre + r0;
    const hipError_t e = a.H % 8 ? (a.x_bf16 ? norm_forward_t<true, true>(p, s) : norm_forward_t<false, true>(p, s))
                                 : (a.x_bf16 ? norm_forward_t<true, false>(p, s) : norm_forward_t<false, false>(p, s));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s) {
  if (a.H % 8) return a.x_bf16 ? norm_backward_t<true, true>(a, s) : norm_backward_t<false, true>(a, s);
  return a.x_bf16 ? norm_backward_t<true, false>(a, s) : norm_backward_t<false, false>(a, s);
}

}  // namespace nf4moe
