// The losses of a vocabulary head, softmax cross entropy and distillation from a teacher's top
// logits, without ever storing the logits l = x W^T [T, V].
//
// Forward: a tile of logits is reduced in registers to a maximum and a sum of exponentials a row
// (k_head_stats), the tiles' pairs are joined row by row (k_head_join):
//   lse = log sum_v exp(l_v / tau);  CE: loss = lse - l_label
//   distillation: q = softmax of the teacher's given logits / tau (k_head_teacher),
//   loss = tau^2 sum_j q_j (log q_j - l_{id_j} / tau + lse)
// The logits that the loss names are picked out of the tile that holds them.
// Backward, by pieces of the vocabulary that the last-level cache can hold: the tile's logits again,
//   P = dloss (exp(l - lse) - [v is the label])         or dloss tau (softmax - q)
// rounded to bf16 (half a step of 2^-8 of each value, no more than the gradients' own
// rounding; P is the operand of two bf16 products), then dx += P W and dW = P^T x.
// All of it is bound by the matrix cores; a handful of rows by the reading of W.
//
// Exponentials are taken in powers of two: z = l log2(e) / tau.
#include "dense.h"
#include "gemm16.h"
#include "internal.h"

namespace nf4moe {

namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kLowest = -3.402823466e38f;

// Adds (m2, s2) to (m, s): sums of 2^(z - m). m may be -inf with s = 0.
__device__ inline void join_stats(float &m, float &s, float m2, float s2) {
  const float top = fmaxf(fmaxf(m, m2), kLowest);
  s = s * __builtin_amdgcn_exp2f(m - top) + s2 * __builtin_amdgcn_exp2f(m2 - top);
  m = top;
}

// A wave's block row mb of logits (16 rows, 16 NB columns) as fp32 rows in its own part of LDS.
template <class T>
struct Staged {
  static constexpr int PITCH = 16 * T::NB * 4 + 16, BYTES = 16 * PITCH;   // rows 4 banks apart
  static constexpr int LDS = BYTES * T::WM * T::WN;
};

template <class T, bool TEACH>
__global__ __launch_bounds__(T::THREADS) void k_head_stats(HeadArgs p) {
  constexpr int SIZE = TEACH && Staged<T>::LDS > T::LDS ? Staged<T>::LDS : T::LDS;
  __shared__ __attribute__((aligned(16))) char lds[SIZE];
  const int mt = (int)((p.T + T::BM - 1) / T::BM), nt = (int)((p.V + T::BN - 1) / T::BN);
  int tm, tn;
  if (!gemm_tile_of(blockIdx.x, mt, nt, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
  T t;
  t.x.init(p.x, p.H, m0, p.T);
  t.y.init(p.w, p.H, n0, p.V);
  t.run(lds, 0, p.H, nullptr);
  const int wn = T::wave_n(), wave = (int)threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int left = (int)(p.V - n0 < T::BN ? p.V - n0 : T::BN);   // columns that exist
  const float c = kLog2e / p.tau;
  float ms[T::MB], ss[T::MB];
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb) {
    const int64_t row = m0 + T::row_of(mb);
    if constexpr (!TEACH) {   // the label's logit, by the one lane that has it
      int want = -1;
      if (row < p.T) {
        const int64_t at = (int64_t)p.ids[row] - n0;
        want = at >= 0 && at < left ? (int)at : -1;
      }
      float got = 0.0f;
      bool here = false;
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool hit = want == T::col_of(nb) + i;
          got = hit ? t.acc[nb][mb][i] : got;
          here |= hit;
        }
      if (here) p.picked[row] = got;
    } else {
      // rows of fp32 in the wave's own part of LDS; its lanes look the entries' ids through
      char *mine = lds + wave * Staged<T>::BYTES;
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb) {
        const f32x4_t &v = t.acc[nb][mb];
        *reinterpret_cast<float4 *>(mine + (lane & 15) * Staged<T>::PITCH + 4 * (nb * 16 + 4 * (lane >> 4))) =
            make_float4(v[0], v[1], v[2], v[3]);
      }
      lds_barrier();
      const int64_t r0 = m0 + (T::wave_m() * T::MB + mb) * 16;
      const int rows = (int)(p.T - r0 < 16 ? p.T - r0 : 16), first = wn * 16 * T::NB;
      const int last = left < first + 16 * T::NB ? left : first + 16 * T::NB;
      for (int e = lane; e < rows * p.k; e += 64) {
        const int64_t at = (int64_t)p.ids[r0 * p.k + e] - n0;
        if (at >= first && at < last)
          p.logits[r0 * p.k + e] = *reinterpret_cast<const float *>(mine + e / p.k * Staged<T>::PITCH + 4 * (at - first));
      }
      lds_barrier();
    }
    float m = -__builtin_inff();
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = T::col_of(nb) + i < left ? t.acc[nb][mb][i] * c : -__builtin_inff();
        t.acc[nb][mb][i] = z;
        m = fmaxf(m, z);
      }
    const float top = fmaxf(m, kLowest);
    float s = 0.0f;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) s += __builtin_amdgcn_exp2f(t.acc[nb][mb][i] - top);
    join_stats(m, s, __shfl_xor(m, 16, kWave), __shfl_xor(s, 16, kWave));
    join_stats(m, s, __shfl_xor(m, 32, kWave), __shfl_xor(s, 32, kWave));
    ms[mb] = m, ss[mb] = s;
  }
  // the waves of a row, in order
  float2 *red = reinterpret_cast<float2 *>(lds);
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb)
    if (lane < 16) red[wn * T::BM + T::row_of(mb)] = make_float2(ms[mb], ss[mb]);
  lds_barrier();
  for (int r = threadIdx.x; r < T::BM; r += T::THREADS) {
    if (m0 + r >= p.T) continue;
    float2 v = red[r];
    for (int w = 1; w < T::WN; ++w) join_stats(v.x, v.y, red[w * T::BM + r].x, red[w * T::BM + r].y);
    p.stats[(int64_t)tn * p.T + m0 + r] = v;
  }
}

// A wave a row: q [k] from the teacher's logits. Entries outside the vocabulary count for
// nothing, an id's later occurrences add to its first; a row without a finite entry has all zeros.
// Also zeros the picked logits of entries outside.
__global__ __launch_bounds__(256) void k_head_teacher(HeadArgs p) {
  __shared__ float val[4][kMaxTeacher];
  __shared__ int32_t ids[4][kMaxTeacher];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + w;
  const bool live = row < p.T;
  const int64_t base = (live ? row : 0) * p.k;
  float m = -__builtin_inff();
  bool nan = false;
  for (int j = lane; j < p.k; j += 64) {
    int32_t id = p.ids[base + j];
    float t = p.teacher_bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p.teacher)[base + j])
                             : reinterpret_cast<const float *>(p.teacher)[base + j];
    if (id < 0 || id >= p.V) {
      id = -1, t = -__builtin_inff();
      if (live) p.logits[base + j] = 0.0f;
    }
    ids[w][j] = id, val[w][j] = t;
    nan |= t != t;
    m = fmaxf(m, t);
  }
  m = wave_max(m);
  nan = __any(nan);
  float sum = 0.0f;
  for (int j = lane; j < p.k; j += 64) {
    const float e = m == -__builtin_inff() ? 0.0f : expf((val[w][j] - m) / p.tau);
    val[w][j] = e;
    sum += e;
  }
  sum = wave_sum(sum);
  lds_barrier();
  if (!live) return;
  for (int j = lane; j < p.k; j += 64) {
    const int32_t id = ids[w][j];
    float e = 0.0f;
    bool first = id >= 0;
    if (first) {
      for (int i = 0; i < p.k; ++i) {
        if (ids[w][i] != id) continue;
        if (i < j) first = false;
        e += val[w][i];
      }
    }
    p.q[base + j] = nan && id >= 0 ? __builtin_nanf("") : first && m != -__builtin_inff() ? e / sum : 0.0f;
  }
}

// 16 rows a workgroup, 16 threads each: the tiles' pairs to lse, and the loss.
__global__ __launch_bounds__(256) void k_head_join(HeadArgs p, int nt) {
  __shared__ float2 red[16][17];
  __shared__ float row_lse[16];
  const int r = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + r;
  const bool live = row < p.T;
  float m = -__builtin_inff(), s = 0.0f;
  if (live) {
#pragma unroll 4
    for (int n = part; n < nt; n += 16) {
      const float2 v = p.stats[(int64_t)n * p.T + row];
      join_stats(m, s, v.x, v.y);
    }
  }
  red[part][r] = make_float2(m, s);
  lds_barrier();
  if (part == 0) {
    for (int i = 1; i < 16; ++i) join_stats(m, s, red[i][r].x, red[i][r].y);
    row_lse[r] = (m + log2f(s)) * kLn2;
  }
  lds_barrier();
  const float lse = row_lse[r];
  if (p.k == 0) {
    if (part == 0 && live) {
      const int32_t id = p.ids[row];
      p.loss[row] = id >= 0 && id < p.V ? lse - p.picked[row] : 0.0f;
      p.lse[row] = lse;
    }
    return;
  }
  float sum = 0.0f, any = 0.0f;
  if (live) {
    for (int j = part; j < p.k; j += 16) {
      const float q = p.q[row * p.k + j];
      if (q == 0.0f) continue;
      any = 1.0f;
      sum += q * (logf(q) - p.logits[row * p.k + j] / p.tau + lse);
    }
  }
  lds_barrier();
  red[part][r] = make_float2(sum, any);
  lds_barrier();
  if (part == 0 && live) {
    for (int i = 1; i < 16; ++i) sum += red[i][r].x, any += red[i][r].y;
    p.loss[row] = any != 0.0f ? p.tau * p.tau * sum : 0.0f;
    p.lse[row] = any != 0.0f ? lse : __builtin_inff();
  }
}

// Whether a row has a gradient: a label in the vocabulary; an lse that is not the +inf of a row
// without teacher entries.
__device__ inline bool row_on(const HeadArgs &p, int64_t row) {
  if (p.k) return p.lse[row] != __builtin_inff();
  const int32_t id = p.ids[row];
  return id >= 0 && id < p.V;
}

// A wave 64 rows.
__global__ __launch_bounds__(256) void k_head_live(HeadArgs p) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const uint64_t bits = __ballot(row < p.T && row_on(p, row));
  if ((threadIdx.x & 63) == 0 && row < p.T) p.live[row >> 6] = bits;
}

template <class T, bool TEACH>
__global__ __launch_bounds__(T::THREADS) void k_head_piece(HeadArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int mt = (int)((p.T + T::BM - 1) / T::BM), nt = (int)((p.vn + T::BN - 1) / T::BN);
  int tm, tn;
  if (!gemm_tile_of(blockIdx.x, mt, nt, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;   // column of the piece
  T t;
  t.x.init(p.x, p.H, m0, p.T);
  t.y.init(p.w + p.v0 * p.H, p.H, n0, p.vn);
  t.run(lds, 0, p.H, nullptr);
  const int left = (int)(p.vn - n0 < T::BN ? p.vn - n0 : T::BN);
  const float c = kLog2e / p.tau;
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb) {
    const int r = T::row_of(mb);
    const int64_t row = m0 + r;
    const bool on = row < p.T && row_on(p, row);
    const float coef = on ? p.dloss[row] * p.tau : 0.0f, lse = on ? p.lse[row] * kLog2e : 0.0f;
    int64_t want = -1;
    if (!TEACH && on) want = (int64_t)p.ids[row] - p.v0 - n0;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = T::col_of(nb) + j;
        float d = __builtin_amdgcn_exp2f(t.acc[nb][mb][j] * c - lse);
        if (!TEACH) d -= want == n ? 1.0f : 0.0f;
        v[j] = on && n < left ? coef * d : 0.0f;
      }
      *reinterpret_cast<uint2 *>(lds + r * T::PITCH + 2 * T::col_of(nb)) = pack4(v[0], v[1], v[2], v[3]);
    }
  }
  lds_barrier();
  if constexpr (TEACH) {   // the entries' places, from their logits in fp32
    const int64_t rows = p.T - m0 < T::BM ? p.T - m0 : T::BM;
    for (int64_t e = threadIdx.x; e < rows * p.k; e += T::THREADS) {
      const int64_t at = (int64_t)p.ids[m0 * p.k + e] - p.v0 - n0;
      if (at < 0 || at >= left) continue;
      const float q = p.q[m0 * p.k + e];
      const int r = (int)(e / p.k);
      if (q == 0.0f || !row_on(p, m0 + r)) continue;
      const float d = __builtin_amdgcn_exp2f(p.logits[m0 * p.k + e] * c - p.lse[m0 + r] * kLog2e) - q;
      *reinterpret_cast<uint16_t *>(lds + r * T::PITCH + 2 * at) = (uint16_t)f32_to_bf16_rne(p.dloss[m0 + r] * p.tau * d);
    }
    lds_barrier();
  }
  store_tile<T::BM, T::BN, T::THREADS>(lds, T::PITCH, p.P + m0 * p.vp + n0, p.vp, p.T - m0, p.vp - n0);
}

// The tile of a call: the largest that gives most of the CUs one.
struct HeadTile {
  int bm, bn;
};
HeadTile head_tile(int64_t T, int64_t V) {
  if (cdiv(T, 256) * cdiv(V, 256) >= 160 && T > 128) return {256, 256};
  if (cdiv(T, 128) * cdiv(V, 128) >= 160 && T > 32) return {128, 128};
  if (T > 32) return {64, 64};
  return {32, 64};
}

template <class F>
void by_head_tile(HeadTile t, F &&f) {
  if (t.bm == 256) f(GemmTile<4, 8, 4, 2>());
  else if (t.bm == 128) f(GemmTile<4, 4, 2, 2>());
  else if (t.bm == 64) f(GemmTile<2, 2, 2, 2>());
  else f(GemmTile<2, 2, 1, 2>());
}

}  // namespace

int64_t head_stat_tiles(int64_t T, int64_t V) { return cdiv(V, head_tile(T, V).bn); }

hipError_t launch_head_forward(const HeadArgs &a, hipStream_t s) {
  if (a.k) {
    hipLaunchKernelGGL(k_head_teacher, dim3((unsigned)cdiv(a.T, 4)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const HeadTile ht = head_tile(a.T, a.V);
  by_head_tile(ht, [&](auto tile) {
    using T = decltype(tile);
    const dim3 grid(gemm_grid(cdiv(a.T, T::BM), cdiv(a.V, T::BN)));
    if (a.k) hipLaunchKernelGGL((k_head_stats<T, true>), grid, dim3(T::THREADS), 0, s, a);
    else hipLaunchKernelGGL((k_head_stats<T, false>), grid, dim3(T::THREADS), 0, s, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_head_join, dim3((unsigned)cdiv(a.T, 16)), dim3(256), 0, s, a, (int)cdiv(a.V, ht.bn));
  return hipGetLastError();
}

hipError_t launch_head_live(const HeadArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(k_head_live, dim3((unsigned)cdiv(a.T, 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_head_piece(const HeadArgs &a, hipStream_t s) {
  by_head_tile(head_tile(a.T, a.vn), [&](auto tile) {
    using T = decltype(tile);
    const dim3 grid(gemm_grid(cdiv(a.T, T::BM), cdiv(a.vn, T::BN)));
    if (a.k) hipLaunchKernelGGL((k_head_piece<T, true>), grid, dim3(T::THREADS), 0, s, a);
    else hipLaunchKernelGGL((k_head_piece<T, false>), grid, dim3(T::THREADS), 0, s, a);
  });
  return hipGetLastError();
}

// Columns of a piece: P [T, piece] in bf16 takes at most 128 MB of the 256 MB last-level cache, so that
// the two products read it from there; whole rounds of 256 tiles where T allows (4096 columns for
// 4096 rows), at least 256.
int64_t head_piece(int64_t T, int64_t V) {
  int64_t n = ((int64_t)1 << 26) / (T > 0 ? T : 1);
  if (n >= V) return (V + 255) / 256 * 256;
  n = n >= 4096 ? n / 4096 * 4096 : n / 256 * 256;
  return n < 256 ? 256 : n;
}

}  // namespace nf4moe
