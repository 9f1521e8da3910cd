// The gated feed-forward of dense bf16 weights (a shared expert's gate and up half), and the products
// that the backward passes of the dense operators share.
//
// Forward: g = x Wg^T, u = x Wu^T, h = act(g, u) in one kernel: a tile takes the gate and
// the up rows of the same columns in alternating groups, so a lane holds g and u of the same
// places and the activation needs no exchange; neither g nor u reaches memory.
// Backward: the same product again, dgu = dh through the activation written in w13's row
// order, then dx = dgu W13 and dW13 = dgu^T x in one launch, which read W13 and x as they lie
// (gemm16.h's turned sides). dgu is rounded to bf16, half a step of 2^-8 of each value, because it is an
// operand of bf16 products; up to kTwoParts rows it is held in two parts, which leave 2^-17.
//
// Measured, us: forward of 4096 rows, H 2048, I 8192 210 to 213 (1290 to 1310 TFLOP/s; the bare products by a
// library 198), of 4099, H = I = 2880 108 to 115 (1180 to 1260, 5 % more in its padding); backward of
// the first 645 to 683 (1210 to 1280 of 825 GFLOP). All of these are bound by the matrix cores and their
// power. One row, H 2048, I 1024: 5.2, of which the 8.4 MB of weights would take 1.6: a launch's
// latency and memory's; 32 rows, H 4096, I 14336 45 to 47 for 235 MB (5.0 to 5.2 TB/s). 131 rows, H 2048, I 768,
// backward: 24.4 for 10 (gate, up, dgu) + 13 (products) + 4 (dx's slices joined), the latencies of
// three dependent launches.
#include "dense.h"
#include "gemm16.h"
#include "internal.h"

namespace nf4moe {

namespace {

// The clamps by comparisons, which a NaN passes through (the minimum of a NaN and a limit is the limit).
__device__ inline float not_above(float v, float limit) { return v > limit ? limit : v; }
__device__ inline float within(float v, float limit) { return not_above(v < -limit ? -limit : v, limit); }

// h from gate and up, as glu_value.
__device__ inline float glu_of(int glu, float alpha, float limit, float g, float u) {
  if (glu == 1) return (within(u, limit) + 1.0f) * sig_gate(not_above(g, limit), alpha);
  return sig_gate(g, 1.0f) * u;
}
// The same, and the activation's derivatives by gate and up. The clamped form's gradient is that of the
// unclamped side at the limit itself.
__device__ inline float glu_slopes(int glu, float alpha, float limit, float g, float u, float &by_g, float &by_u) {
  const bool clamped = glu == 1;
  const float a = clamped ? alpha : 1.0f;
  const float gc = clamped ? not_above(g, limit) : g;
  const float uc = clamped ? within(u, limit) + 1.0f : u;
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gc * (-1.44269504088896341f * a)));
  const float gs = gc * s;
  by_u = clamped && fabsf(u) > limit ? 0.0f : gs;
  by_g = clamped && g > limit ? 0.0f : uc * (s + a * gs * (1.0f - s));
  return uc * gs;
}

template <class T>
struct FfnPlace : GemmTiles {
  const FfnArgs &p;
  __device__ FfnPlace(const FfnArgs &a, int b, int nb)
      : GemmTiles{b, nb, (int)((a.T + T::BM - 1) / T::BM), (a.I + T::BN / 2 - 1) / (T::BN / 2), 1, a.H}, p(a) {}
  __device__ bool at(int r, int64_t &m0, int64_t &c0) const {
    int m, n, slice;
    if (!find(r, m, n, slice)) return false;
    m0 = (int64_t)m * T::BM, c0 = (int64_t)n * (T::BN / 2);
    return true;
  }
  __device__ bool operator()(int r, typename T::X &x, typename T::Y &y, GemmRange &k) const {
    int64_t m0, c0;
    if (!at(r, m0, c0)) return false;
    x.init(p.x, p.H, m0, p.T);
    y.template init_pair<T::G>(p.w13, p.w13 + (p.inter ? 1 : (int64_t)p.I) * p.H, (p.inter ? 2 : 1) * (int64_t)p.H, c0, p.I);
    k = {0, p.H};
    return true;
  }
};

// BACK: dgu (and h where asked for) instead of h. FEW: up to kTwoParts rows, dgu in two parts and x twice.
template <class T, bool BACK, bool FEW>
__global__ __launch_bounds__(T::THREADS, T::WAVES_SIMD) void k_ffn(FfnArgs p) {
  static_assert(BACK || !FEW, "two parts of what a backward rounds");
  constexpr int G = T::G, HC = 16 * G;   // a wave's columns of h
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  if constexpr (FEW) {
    const int n = (int)p.T * (p.H / 8);   // 16-byte pieces
    for (int i = (int)blockIdx.x * T::THREADS + threadIdx.x; p.x2 && i < n; i += (int)gridDim.x * T::THREADS) {
      const uint4 v = reinterpret_cast<const uint4 *>(p.x)[i];
      reinterpret_cast<uint4 *>(p.x2)[i] = v;
      reinterpret_cast<uint4 *>(p.x2)[n + i] = v;
    }
  }
  const FfnPlace<T> place(p, blockIdx.x, gridDim.x);
  int64_t m0, c0;
  if (!place.at(0, m0, c0)) return;
  T t;
  t.run(lds, nullptr, place, [&](int r) __attribute__((always_inline)) {
    place.at(r, m0, c0);
    c0 += T::wave_n() * HC;
    char *mine = T::scratch(lds);
    const int lane = epilogue_lane();
    const int64_t cols = p.I - c0, ld2 = 2 * (int64_t)p.I;
    [[maybe_unused]] uint2 d[T::MB][G];
    if constexpr (BACK) {   // asked for together
#pragma unroll
      for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < G; ++nb) {
          const int64_t row = m0 + T::row_at(mb) + (lane & 15);
          d[mb][nb] = make_uint2(0, 0);
          if (row < p.T && T::col_of(lane, nb) < cols) d[mb][nb] = *reinterpret_cast<const uint2 *>(p.dh + row * p.I + c0 + T::col_of(lane, nb));
        }
    }
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int64_t row0 = m0 + T::row_at(mb), rows = p.T - row0;
      if (rows <= 0) break;   // the wave
      if constexpr (!BACK) {
        const BlockRow<HC> out{mine, lane};
#pragma unroll
        for (int nb = 0; nb < G; ++nb) {
          float h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = glu_of(p.glu, p.alpha, p.limit, t.acc[nb][mb][j], t.acc[nb + G][mb][j]);
          out.put(T::col_of(lane, nb), pack4(h[0], h[1], h[2], h[3]));
        }
        out.out(p.h + row0 * p.I + c0, p.I, rows, cols);
      } else {
        const BlockRow<HC> one{mine, lane}, two{mine + 32 * HC, lane};
        const BlockRow<2 * HC> both{mine, lane};
        uint2 h[G];
        [[maybe_unused]] float low[2][FEW ? G : 1][4];
        auto put = [&](int nb, const float (&dg)[4], const float (&du)[4]) __attribute__((always_inline)) {
          const int c = T::col_of(lane, nb);
          if (p.inter) {
            both.put(2 * c, pack4(dg[0], du[0], dg[1], du[1]));
            both.put(2 * c + 4, pack4(dg[2], du[2], dg[3], du[3]));
          } else {
            one.put(c, pack4(dg[0], dg[1], dg[2], dg[3]));
            two.put(c, pack4(du[0], du[1], du[2], du[3]));
          }
        };
        auto out = [&](int64_t first) __attribute__((always_inline)) {
          uint16_t *dgu = p.dgu + (first + row0) * ld2;
          if (p.inter) {
            both.out(dgu + 2 * c0, ld2, rows, 2 * cols);
          } else {
            one.out(dgu + c0, ld2, rows, cols);
            two.out(dgu + p.I + c0, ld2, rows, cols);
          }
        };
#pragma unroll
        for (int nb = 0; nb < G; ++nb) {
          const float dh[4] = {bf16lo_to_f32(d[mb][nb].x), bf16hi_to_f32(d[mb][nb].x), bf16lo_to_f32(d[mb][nb].y), bf16hi_to_f32(d[mb][nb].y)};
          float dg[4], du[4], hv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float by_g, by_u;
            hv[j] = glu_slopes(p.glu, p.alpha, p.limit, t.acc[nb][mb][j], t.acc[nb + G][mb][j], by_g, by_u);
            dg[j] = dh[j] * by_g, du[j] = dh[j] * by_u;
            if constexpr (FEW) {
              low[0][nb][j] = bf16_rest(dg[j]);
              low[1][nb][j] = bf16_rest(du[j]);
            }
          }
          h[nb] = pack4(hv[0], hv[1], hv[2], hv[3]);
          put(nb, dg, du);
        }
        out(0);
        if constexpr (FEW) {
#pragma unroll
          for (int nb = 0; nb < G; ++nb) put(nb, low[0][nb], low[1][nb]);
          out(p.T);
        }
        if (p.h) {
#pragma unroll
          for (int nb = 0; nb < G; ++nb) one.put(T::col_of(lane, nb), h[nb]);
          one.out(p.h + row0 * p.I + c0, p.I, rows, cols);
        }
      }
    }
  });
}

// Up to 16 tokens: a workgroup takes eight gate rows and their up rows.
__global__ __launch_bounds__(512) void k_ffn_few(FfnArgs p) {
  using F = FewRows<8>;
  __shared__ __attribute__((aligned(16))) char lds[F::LDS];
  const int c0 = (int)blockIdx.x * 8, T = (int)p.T;
  f32x4_t v = F::run(
      lds, p.H,
      [&](int i) {
        const int64_t c = c0 + (i & 7);
        return p.w13 + (p.inter ? 2 * c + (i >> 3) : c + (i >> 3) * (int64_t)p.I) * p.H;
      },
      [&](int i) { return p.x + (int64_t)(i < T ? i : T - 1) * p.H; });
  const int lane = threadIdx.x & 63, token = lane & 15;
  if (threadIdx.x >= 64) return;
  float h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = glu_of(p.glu, p.alpha, p.limit, v[j], __shfl_xor(v[j], 32, kWave));   // (lanes 0 .. 31: the gate rows)
  if (lane < 32 && token < T)
    *reinterpret_cast<uint2 *>(p.h + (int64_t)token * p.I + c0 + 4 * (lane >> 4)) = pack4(h[0], h[1], h[2], h[3]);
}

// Up to 32 tokens, many columns: a workgroup takes 32 gate rows and their up rows, a wave 16 of each for 16 tokens.
__global__ __launch_bounds__(256) void k_ffn_stream(FfnArgs p) {
  using F = FewStream<6, 2>;   // (144 KB for two workgroups a CU)
  __shared__ __attribute__((aligned(16))) char lds[F::LDS];
  const int64_t c0 = (int64_t)blockIdx.x * 32;
  typename F::X x;
  typename F::Y y;
  x.init(p.x, p.H, 0, p.T);
  y.template init_pair<2>(p.w13, p.w13 + (p.inter ? 1 : (int64_t)p.I) * p.H, (p.inter ? 2 : 1) * (int64_t)p.H, c0, p.I);
  const int wave = F::X::wave(), lane = threadIdx.x & 63, nb = wave & 1, mb = wave >> 1;
  f32x4_t g = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, u = g;
  const bool mine = 16 * mb < p.T;   // the wave
  F::run(lds, p.H, x, y, [&](const char *xs, const char *ys) __attribute__((always_inline)) {
    if (!mine) return;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const bf16x8_t fx = F::X::frag(xs, mb, kk);
      g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(F::Y::frag(ys, nb, kk), fx, g, 0, 0, 0);
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(F::Y::frag(ys, nb + 2, kk), fx, u, 0, 0, 0);
    }
  });
  const int64_t token = 16 * mb + (lane & 15), col = c0 + 16 * nb + 4 * (lane >> 4);
  if (token >= p.T || col >= p.I) return;
  float h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = glu_of(p.glu, p.alpha, p.limit, g[j], u[j]);
  *reinterpret_cast<uint2 *>(p.h + token * p.I + col) = pack4(h[0], h[1], h[2], h[3]);
}

template <class T>
struct ProductPlace : GemmTiles {
  const ProductArgs &p;
  __device__ ProductPlace(const ProductArgs &a, int b, int nb, int log)
      : GemmTiles{b, nb, (int)((a.M + T::BM - 1) / T::BM), (int)((a.N + T::BN - 1) / T::BN), a.slices, a.K, log}, p(a) {}
  __device__ bool operator()(int r, typename T::X &x, typename T::Y &y, GemmRange &k) const {
    int m, n, slice;
    if (!find(r, m, n, slice)) return false;
    x.init(p.x, p.ldx, (int64_t)m * T::BM, p.M);
    y.init(p.y, p.ldy, (int64_t)n * T::BN, p.N);
    k = range_of(slice);
    return true;
  }
};

// The tiles of workgroup b of nb of a product. UNIT: outputs times *unit_at, one argument for both products, read where
// it is used (in each product's arguments its address took 23 scalar registers more, spilled in the steps' loop,
// and 1 to 2 %).
template <class T, bool UNIT>
__device__ __attribute__((always_inline)) void product_tiles(const ProductArgs &p, const float *unit_at, char *lds, int b, int nb, int log = 3) {
  const ProductPlace<T> place(p, b, nb, log);
  int m, n, slice;
  if (!place.find(0, m, n, slice)) return;
  T t;
  t.run(lds, p.live, place, [&](int r) __attribute__((always_inline)) {
    place.find(r, m, n, slice);
    const int64_t n0 = (int64_t)n * T::BN + T::cols_at(), cols = p.N - n0;
    if (cols <= 0) return;   // the wave
    float *part = p.part + (int64_t)slice * p.M * p.N;
    const int lane = epilogue_lane();
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int64_t row0 = (int64_t)m * T::BM + T::row_at(mb), rows = p.M - row0;
      if (rows <= 0) break;   // the wave
      if (p.out) {
        const float unit = UNIT ? *unit_at : 1.0f;
        const BlockRow<16 * T::NB> out{T::scratch(lds), lane};
#pragma unroll
        for (int nb2 = 0; nb2 < T::NB; ++nb2) {
          const f32x4_t v = UNIT ? t.acc[nb2][mb] * unit : t.acc[nb2][mb];
          out.put(T::col_of(lane, nb2), pack4(v[0], v[1], v[2], v[3]));
        }
        out.out(p.out + row0 * p.N + n0, p.N, rows, cols);
        continue;
      }
      if ((lane & 15) >= rows) continue;
      float *at = part + (row0 + (lane & 15)) * p.N + n0;
      float4 was[T::NB];
      if (p.add) {
#pragma unroll
        for (int nb2 = 0; nb2 < T::NB; ++nb2)
          if (T::col_of(lane, nb2) < cols) was[nb2] = *reinterpret_cast<const float4 *>(at + T::col_of(lane, nb2));
      } else {
#pragma unroll
        for (int nb2 = 0; nb2 < T::NB; ++nb2) was[nb2] = make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int nb2 = 0; nb2 < T::NB; ++nb2) {
        const f32x4_t &v = t.acc[nb2][mb];
        if (T::col_of(lane, nb2) < cols)
          *reinterpret_cast<float4 *>(at + T::col_of(lane, nb2)) =
              make_float4(was[nb2].x + v[0], was[nb2].y + v[1], was[nb2].z + v[2], was[nb2].w + v[3]);
      }
    }
  });
}

// Workgroups 0 .. nbx - 1 take dx's tiles, the others dw's: side by side they fill the card together, where
// dx by itself has its k in slices to be joined (4096 rows, H 2048, I 8192: dx 198 us alone and 13 to
// join, dw 200, both 392).
// nbx < 0, for large products of equal steps: half of the XCDs each, so that an L2 holds the operands
// of one product (1 to 1.7 % of a whole backward).
template <class TX, class TW, bool UNIT>
__global__ __launch_bounds__(TX::THREADS, TX::WAVES_SIMD) void k_products(ProductArgs dx, ProductArgs dw, const float *unit_at, int nbx) {
  static_assert(TX::THREADS == TW::THREADS, "one workgroup size");
  __shared__ __attribute__((aligned(16))) char lds[TX::LDS > TW::LDS ? TX::LDS : TW::LDS];
  const int b = blockIdx.x, nb = gridDim.x;
  if (nbx < 0) {   // half of the XCDs each
    const int half = (b >> 3) * 4 + (b & 3);
    if ((b & 7) < 4) product_tiles<TX, UNIT>(dx, unit_at, lds, half, nb / 2, 2);
    else product_tiles<TW, UNIT>(dw, unit_at, lds, half, nb / 2, 2);
    return;
  }
  if (b < nbx) product_tiles<TX, UNIT>(dx, unit_at, lds, b, nbx);
  else product_tiles<TW, UNIT>(dw, unit_at, lds, b - nbx, nb - nbx);
}

// Few slices: 8 values a thread at a time, n a multiple of 8.
__global__ __launch_bounds__(256) void k_join(const float *part, int slices, int64_t n, const float *unit, uint16_t *out) {
  const float by = unit ? *unit : 1.0f;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    float4 a = make_float4(0, 0, 0, 0), b = a;
    for (int s = 0; s < slices; ++s) {
      const float4 *at = reinterpret_cast<const float4 *>(part + s * n + i);
      const float4 u = at[0], v = at[1];
      a = make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w);
      b = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
    }
    const uint2 lo = pack4(a.x * by, a.y * by, a.z * by, a.w * by), hi = pack4(b.x * by, b.y * by, b.z * by, b.w * by);
    *reinterpret_cast<uint4 *>(out + i) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}
// Many: a workgroup 256 values at a time, wave w the slices w, w + 8, .. in order, asked for eight together;
// then the waves in order. (128 slices of 3168 values: 19 us by k_join, two workgroups with 128 trips to
// memory each, 4 by this.)
__global__ __launch_bounds__(512) void k_join_many(const float *part, int slices, int64_t n, const float *unit, uint16_t *out) {
  __shared__ float4 red[8][64];
  const float by = unit ? *unit : 1.0f;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < n; i0 += (int64_t)gridDim.x * 256) {
    const int64_t i = i0 + 4 * lane;
    float4 a = make_float4(0, 0, 0, 0);
    if (i < n) {
#pragma unroll 8
      for (int s = wave; s < slices; s += 8) {
        const float4 v = *reinterpret_cast<const float4 *>(part + s * n + i);
        a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
      }
    }
    red[wave][lane] = a;
    lds_barrier();
    if (wave == 0 && i < n) {
#pragma unroll
      for (int w = 1; w < 8; ++w) {
        const float4 v = red[w][lane];
        a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
      }
      *reinterpret_cast<uint2 *>(out + i) = pack4(a.x * by, a.y * by, a.z * by, a.w * by);
    }
    lds_barrier();
  }
}

int64_t ffn_tile_count(const void *args, int bm, int bn) {
  const FfnArgs &a = *static_cast<const FfnArgs *>(args);
  return cdiv(a.T, bm) * cdiv(a.I, bn / 2);
}

template <bool BACK>
hipError_t ffn(const FfnArgs &a, hipStream_t s) {
  auto go = [&](auto tile) {
    using T = typename decltype(tile)::type;
    const int64_t tiles = cdiv(a.T, T::BM) * cdiv(a.I, T::BN / 2);
    const int grid = T::KS > 1 ? (int)cdiv(tiles, 8) * 8 : gemm_grid(tiles, T::MOST);
    if constexpr (BACK && T::BM <= 64) {   // (the tiles of few rows)
      if (a.T <= kTwoParts) {
        hipLaunchKernelGGL((k_ffn<T, true, true>), dim3(grid), dim3(T::THREADS), 0, s, a);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((k_ffn<T, BACK, false>), dim3(grid), dim3(T::THREADS), 0, s, a);
    return hipGetLastError();
  };
  int c = gemm_class(ffn_tile_count, &a, cdiv(a.H, kGemmBK));
  if (a.T <= kTwoParts && c > 64) c = 64;
  switch (c) {
    case 256: return go(TileTag<GemmTile<4, 8, 4, 2, false, false, 4>>());
    case 192: return go(TileTag<GemmTile<3, 8, 4, 2, false, false, 4>>());
    case 128: return go(TileTag<GemmTile<4, 4, 2, 2, false, false, 2>>());
    case 64: return go(TileTag<GemmTile<2, 4, 2, 1, false, false, 2>>());
    case 16: return go(TileTag<GemmTile<2, 4, 2, 1, false, false, 2, false, 4>>());
    default: return go(TileTag<GemmTile<1, 2, 2, 1, false, false, 1, false, 8>>());
  }
}

struct ProductPair {
  const ProductArgs &x, &w;
};
int64_t product_tile_count(const void *args, int bm, int bn) {
  const ProductPair &a = *static_cast<const ProductPair *>(args);
  const int64_t x = a.x.K ? cdiv(a.x.M, bm) * cdiv(a.x.N, bn) * a.x.slices : 0;
  if (!a.w.K) return x;
  if (bm == 192) return (int64_t)1 << 40;   // (dx alone: a turned side of 192 rows has no whole pieces a thread)
  return x + cdiv(a.w.M, bm) * cdiv(a.w.N, bn) * a.w.slices;
}

template <class TX, class TW, bool UNIT>
hipError_t products(const ProductArgs &dx, const ProductArgs &dw, const float *unit, hipStream_t s) {
  const int64_t tx = dx.K ? cdiv(dx.M, TX::BM) * cdiv(dx.N, TX::BN) * dx.slices : 0;
  const int64_t tw = dw.K ? cdiv(dw.M, TW::BM) * cdiv(dw.N, TW::BN) * dw.slices : 0;
  int nbx = (int)cdiv(tx, 8) * 8, nbw = (int)cdiv(tw, 8) * 8;
  if (TX::KS == 1 && tx + tw > TX::MOST) {
    // the workgroups that run at a time, shared by the steps that either product takes
    const double sx = (double)tx * (double)cdiv(dx.K, dx.slices ? dx.slices : 1), sw = (double)tw * (double)cdiv(dw.K, dw.slices ? dw.slices : 1);
    const int share = (int)(TX::MOST / 8 * sx / (sx + sw) + 0.5) * 8;
    nbx = !tx ? 0 : !tw ? TX::MOST : share < 8 ? 8 : share > TX::MOST - 8 ? TX::MOST - 8 : share;
    if (tx) nbx = gemm_grid(tx, nbx);
    nbw = tw ? gemm_grid(tw, TX::MOST - nbx) : 0;
  }
  const int split = TX::KS == 1 && nbx == TX::MOST / 2 && nbw == nbx ? -1 : nbx;
  hipLaunchKernelGGL((k_products<TX, TW, UNIT>), dim3(nbx + nbw), dim3(TX::THREADS), 0, s, dx, dw, unit, split);
  return hipGetLastError();
}
template <int MB, int NB, int WM, int WN, bool UNIT, int KS = 1>
hipError_t products_of(const ProductArgs &x, const ProductArgs &w, const float *unit, hipStream_t s) {
  return products<GemmTile<MB, NB, WM, WN, false, true, 0, false, KS>, GemmTile<MB, NB, WM, WN, true, true, 0, UNIT, KS>, UNIT>(x, w, unit, s);
}
// UNIT: those of a vocabulary loss of more than kTwoParts rows, whose outputs have a unit and whose rows for dw a mask.
template <bool UNIT>
hipError_t products(const ProductArgs &x, const ProductArgs &w, const float *unit, hipStream_t s) {
  const ProductPair both{x, w};
  const int64_t steps = cdiv(x.K > w.K ? x.K : w.K, kGemmBK);
  switch (gemm_class(product_tile_count, &both, steps)) {
    case 256: return products_of<4, 8, 4, 2, UNIT>(x, w, unit, s);
    case 192: return products<GemmTile<3, 8, 4, 2, false, true>, GemmTile<4, 8, 4, 2, true, true>, UNIT>(x, w, unit, s);
    case 128: return products_of<4, 4, 2, 2, UNIT>(x, w, unit, s);
    case 64: return products_of<2, 2, 2, 2, UNIT>(x, w, unit, s);
    default: return products_of<2, 2, 2, 2, UNIT, 4>(x, w, unit, s);
  }
}

}  // namespace

hipError_t launch_ffn_forward(const FfnArgs &a, hipStream_t s) {
  // Few rows, in us by tokens, H, I, as few / tiles / stream: 16 2048 1024 7.1 / 8.0 / 10.0; 16 2048 4096 9.9 / 10.4 /
  // 10.2; 1 2048 14336 23.5 / 34 / 25; 8 2048 14336 31 / 34 / 25; 32 4096 4096 28 / 20 / 21; 1 1024 14336 20 / 18 /
  // 12; 16 512 4096 9.8 / 7.6 / 7.7; 16 8192 14336 126 / 130 / 91.
  const bool wide = a.I >= 8192 || (a.H <= 1024 && a.I > 2048);
  if (a.T <= 32 && wide && (a.T > 4 || a.H < 2048))
    hipLaunchKernelGGL(k_ffn_stream, dim3((unsigned)cdiv(a.I, 32)), dim3(256), 0, s, a);
  else if (a.T <= 16)   // (the widest I is 2^20: 2^17 workgroups of 512)
    hipLaunchKernelGGL(k_ffn_few, dim3((unsigned)(a.I / 8)), dim3(512), 0, s, a);
  else
    return ffn<false>(a, s);
  return hipGetLastError();
}
hipError_t launch_ffn_dgu(const FfnArgs &a, hipStream_t s) { return ffn<true>(a, s); }

hipError_t launch_products(const ProductArgs *dx, const ProductArgs *dw, const float *unit, hipStream_t s) {
  const ProductArgs none = {};
  const ProductArgs &x = dx ? *dx : none, &w = dw ? *dw : none;
  return unit ? products<true>(x, w, unit, s) : products<false>(x, w, unit, s);
}

int product_slices(int64_t M, int64_t N, int64_t K, bool alone, int least) {
  const int64_t tiles = cdiv(M, 256) * cdiv(N, 256), steps = cdiv(K, kGemmBK);
  int64_t s = (alone ? 256 : 128) / tiles;
  if (s > steps / least) s = steps / least;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

hipError_t launch_join(const float *part, int slices, int64_t n, const float *unit, uint16_t *out, hipStream_t s) {
  const int64_t g = cdiv(n, slices > 4 ? 256 : 2048), most = 1 << 22;   // (well inside a dispatch's 2^32 threads)
  const dim3 grid((unsigned)(g < most ? g : most));
  if (slices > 4) hipLaunchKernelGGL(k_join_many, grid, dim3(512), 0, s, part, slices, n, unit, out);
  else hipLaunchKernelGGL(k_join, grid, dim3(256), 0, s, part, slices, n, unit, out);
  return hipGetLastError();
}

}  // namespace nf4moe
