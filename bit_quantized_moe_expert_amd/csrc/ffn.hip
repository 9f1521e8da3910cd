// The gated feed-forward block of dense bf16 weights (a shared expert), and the products
// that the backward passes of the dense operators share.
//
// Forward: g = x Wg^T, u = x Wu^T, h = act(g, u) in one kernel: a tile takes the gate and
// the up rows of the same columns in alternating groups, so a lane holds g and u of the same
// places and the activation needs no exchange; neither g nor u reaches memory.
// Backward: the same product again, dgu = dh through the activation written in w13's row
// order, then dx = dgu W13 and dW13 = dgu^T x, which read W13 and x as they lie (gemm16.h's
// turned sides).
#include "dense.h"
#include "gemm16.h"
#include "internal.h"

namespace nf4moe {

namespace {

// h and the activation's derivatives by gate and up. The clamped form's gradient is that of the
// unclamped side at the limit itself.
__device__ inline float glu_slopes(int glu, float alpha, float limit, float g, float u, float &by_g, float &by_u) {
  const bool clamped = glu == 1;
  const float a = clamped ? alpha : 1.0f;
  const float gc = clamped ? fminf(g, limit) : g;
  const float uc = clamped ? fminf(fmaxf(u, -limit), limit) + 1.0f : u;
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gc * (-1.44269504088896341f * a)));
  const float gs = gc * s;
  by_u = clamped && fabsf(u) > limit ? 0.0f : gs;
  by_g = clamped && g > limit ? 0.0f : uc * (s + a * gs * (1.0f - s));
  return uc * gs;
}

// BACK: dgu (and h where asked for) instead of h.
template <class T, bool BACK>
__global__ __launch_bounds__(T::THREADS) void k_ffn(FfnArgs p) {
  constexpr int G = T::G, HN = T::BN / 2;
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int mt = (int)((p.T + T::BM - 1) / T::BM), nt = (p.I + HN - 1) / HN;
  int tm, tn;
  if (!gemm_tile_of(blockIdx.x, mt, nt, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * T::BM, c0 = (int64_t)tn * HN;
  T t;
  t.x.init(p.x, p.H, m0, p.T);
  if (p.inter) t.y.template init_pair<G>(p.w13, p.w13 + p.H, 2 * (int64_t)p.H, c0, p.I);
  else t.y.template init_pair<G>(p.w13, p.w13 + (int64_t)p.I * p.H, p.H, c0, p.I);
  t.run(lds, 0, p.H, nullptr);
  const int wn = T::wave_n(), g4 = 4 * (int)(threadIdx.x >> 4 & 3);
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb) {
    const int r = T::row_of(mb);
    char *row = lds + r * T::PITCH;
#pragma unroll
    for (int nb = 0; nb < G; ++nb) {
      const int c = (wn * G + nb) * 16 + g4;   // column of the tile's HN
      f32x4_t &gv = t.acc[nb][mb], &uv = t.acc[nb + G][mb];
      if constexpr (!BACK) {
        float h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = glu_value(p.glu, p.alpha, p.limit, gv[j], uv[j]);
        *reinterpret_cast<uint2 *>(row + 2 * c) = pack4(h[0], h[1], h[2], h[3]);
      } else {
        uint2 d = make_uint2(0, 0);
        if (m0 + r < p.T && c0 + c < p.I) d = *reinterpret_cast<const uint2 *>(p.dh + (m0 + r) * p.I + c0 + c);
        const float dh[4] = {bf16lo_to_f32(d.x), bf16hi_to_f32(d.x), bf16lo_to_f32(d.y), bf16hi_to_f32(d.y)};
        float dg[4], du[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float by_g, by_u;
          // h takes g's place for the second pass
          gv[j] = glu_slopes(p.glu, p.alpha, p.limit, gv[j], uv[j], by_g, by_u);
          dg[j] = dh[j] * by_g, du[j] = dh[j] * by_u;
        }
        if (p.inter) {
          *reinterpret_cast<uint2 *>(row + 4 * c) = pack4(dg[0], du[0], dg[1], du[1]);
          *reinterpret_cast<uint2 *>(row + 4 * c + 8) = pack4(dg[2], du[2], dg[3], du[3]);
        } else {
          *reinterpret_cast<uint2 *>(row + 2 * c) = pack4(dg[0], dg[1], dg[2], dg[3]);
          *reinterpret_cast<uint2 *>(row + 2 * (HN + c)) = pack4(du[0], du[1], du[2], du[3]);
        }
      }
    }
  }
  lds_barrier();
  const int64_t rows = p.T - m0, cols = p.I - c0;
  if constexpr (!BACK) {
    store_tile<T::BM, HN, T::THREADS>(lds, T::PITCH, p.h + m0 * p.I + c0, p.I, rows, cols);
  } else {
    const int64_t ld = 2 * (int64_t)p.I;
    if (p.inter) {
      store_tile<T::BM, T::BN, T::THREADS>(lds, T::PITCH, p.dgu + m0 * ld + 2 * c0, ld, rows, 2 * cols);
    } else {
      store_tile<T::BM, HN, T::THREADS>(lds, T::PITCH, p.dgu + m0 * ld + c0, ld, rows, cols);
      store_tile<T::BM, HN, T::THREADS>(lds + 2 * HN, T::PITCH, p.dgu + m0 * ld + p.I + c0, ld, rows, cols);
    }
    if (!p.h) return;   // the whole grid
    lds_barrier();
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < G; ++nb) {
        const f32x4_t &h = t.acc[nb][mb];
        *reinterpret_cast<uint2 *>(lds + T::row_of(mb) * T::PITCH + 2 * ((wn * G + nb) * 16 + g4)) = pack4(h[0], h[1], h[2], h[3]);
      }
    lds_barrier();
    store_tile<T::BM, HN, T::THREADS>(lds, T::PITCH, p.h + m0 * p.I + c0, p.I, rows, cols);
  }
}

template <class T>
__global__ __launch_bounds__(T::THREADS) void k_product(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int mt = (int)((p.M + T::BM - 1) / T::BM), nt = (int)((p.N + T::BN - 1) / T::BN);
  int tm, tn;
  if (!gemm_tile_of(blockIdx.x, mt, nt, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
  T t;
  t.x.init(p.x, p.ldx, m0, p.M);
  t.y.init(p.y, p.ldy, n0, p.N);
  // slices of whole steps
  const int64_t steps = (p.K + kGemmBK - 1) / kGemmBK, each = (steps + p.slices - 1) / p.slices;
  const int64_t k0 = blockIdx.y * each * kGemmBK, k1 = k0 + each * kGemmBK < p.K ? k0 + each * kGemmBK : p.K;
  t.run(lds, k0, k1, p.live);
  if (p.out) {
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb) {
        const f32x4_t &v = t.acc[nb][mb];
        *reinterpret_cast<uint2 *>(lds + T::row_of(mb) * T::PITCH + 2 * T::col_of(nb)) = pack4(v[0], v[1], v[2], v[3]);
      }
    lds_barrier();
    store_tile<T::BM, T::BN, T::THREADS>(lds, T::PITCH, p.out + m0 * p.N + n0, p.N, p.M - m0, p.N - n0);
    return;
  }
  float *part = p.part + (int64_t)blockIdx.y * p.M * p.N;
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb) {
    const int64_t m = m0 + T::row_of(mb);
    if (m >= p.M) continue;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
      const int64_t n = n0 + T::col_of(nb);
      if (n >= p.N) continue;
      float4 *at = reinterpret_cast<float4 *>(part + m * p.N + n);
      const f32x4_t &v = t.acc[nb][mb];
      float4 o = make_float4(v[0], v[1], v[2], v[3]);
      if (p.add) {
        const float4 was = *at;
        o = make_float4(was.x + o.x, was.y + o.y, was.z + o.z, was.w + o.w);
      }
      *at = o;
    }
  }
}

// 8 values a thread, n a multiple of 8.
__global__ __launch_bounds__(256) void k_join(const float *part, int slices, int64_t n, uint16_t *out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float4 a = make_float4(0, 0, 0, 0), b = a;
  for (int s = 0; s < slices; ++s) {
    const float4 *at = reinterpret_cast<const float4 *>(part + s * n + i);
    const float4 u = at[0], v = at[1];
    a = make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w);
    b = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
  }
  const uint2 lo = pack4(a.x, a.y, a.z, a.w), hi = pack4(b.x, b.y, b.z, b.w);
  *reinterpret_cast<uint4 *>(out + i) = make_uint4(lo.x, lo.y, hi.x, hi.y);
}

template <bool BACK>
hipError_t ffn(const FfnArgs &a, hipStream_t s) {
  auto tiles = [&](int bm, int hn) { return cdiv(a.T, bm) * cdiv(a.I, hn); };
  if (tiles(256, 128) >= 160) {
    using T = GemmTile<4, 8, 4, 2, false, false, 4>;
    hipLaunchKernelGGL((k_ffn<T, BACK>), dim3(gemm_grid(cdiv(a.T, 256), cdiv(a.I, 128))), dim3(T::THREADS), 0, s, a);
  } else if (tiles(128, 64) >= 160) {
    using T = GemmTile<4, 4, 2, 2, false, false, 2>;
    hipLaunchKernelGGL((k_ffn<T, BACK>), dim3(gemm_grid(cdiv(a.T, 128), cdiv(a.I, 64))), dim3(T::THREADS), 0, s, a);
  } else {
    using T = GemmTile<2, 4, 2, 1, false, false, 2>;
    hipLaunchKernelGGL((k_ffn<T, BACK>), dim3(gemm_grid(cdiv(a.T, 64), cdiv(a.I, 32))), dim3(T::THREADS), 0, s, a);
  }
  return hipGetLastError();
}

template <bool XT, bool MASK>
hipError_t product(const ProductArgs &a, hipStream_t s) {
  auto tiles = [&](int bm, int bn) { return cdiv(a.M, bm) * cdiv(a.N, bn) * a.slices; };
  if (tiles(256, 256) >= 160) {
    using T = GemmTile<4, 8, 4, 2, XT, true, 0, MASK>;
    hipLaunchKernelGGL((k_product<T>), dim3(gemm_grid(cdiv(a.M, 256), cdiv(a.N, 256)), a.slices), dim3(T::THREADS), 0, s, a);
  } else if (tiles(128, 128) >= 160) {
    using T = GemmTile<4, 4, 2, 2, XT, true, 0, MASK>;
    hipLaunchKernelGGL((k_product<T>), dim3(gemm_grid(cdiv(a.M, 128), cdiv(a.N, 128)), a.slices), dim3(T::THREADS), 0, s, a);
  } else {
    using T = GemmTile<2, 2, 2, 2, XT, true, 0, MASK>;
    hipLaunchKernelGGL((k_product<T>), dim3(gemm_grid(cdiv(a.M, 64), cdiv(a.N, 64)), a.slices), dim3(T::THREADS), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s) { return ffn<false>(a, s); }
hipError_t launch_ffn_dgu(const FfnArgs &a, hipStream_t s) { return ffn<true>(a, s); }

hipError_t launch_product(const ProductArgs &a, bool x_turned, hipStream_t s) {
  if (!x_turned) return product<false, false>(a, s);
  return a.live ? product<true, true>(a, s) : product<true, false>(a, s);
}

int product_slices(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = cdiv(M, 256) * cdiv(N, 256), steps = cdiv(K, kGemmBK);
  int64_t s = tiles >= 160 ? 1 : 256 / tiles;
  if (s > steps / 8) s = steps / 8;   // at least 8 steps each
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

hipError_t launch_join(const float *part, int slices, int64_t n, uint16_t *out, hipStream_t s) {
  hipLaunchKernelGGL(k_join, dim3((unsigned)cdiv(n, 2048)), dim3(256), 0, s, part, slices, n, out);
  return hipGetLastError();
}

}  // namespace nf4moe
