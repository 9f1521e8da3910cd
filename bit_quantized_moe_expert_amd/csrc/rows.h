// Rows of any width held by the threads of a workgroup, eight elements a piece: loads, stores
// and sums shared by the norms' kernels.
#pragma once
#include "ckpt8.h"

namespace nf4moe {

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

// Sum over the TPR threads of a row (NV values at once); red has a place per wave and
// value. TPR > 64: one barrier, taken by every thread of the workgroup. Consecutive
// sums use different places (a thread that writes them again has passed another
// sum's barrier, and so has every reader).
template <int TPR, int NV>
__device__ inline void row_sum(float (&v)[NV], float *red) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (TPR >= 64) {
      v[k] = wave_sum(v[k]);
    } else {   // several rows a wave
#pragma unroll
      for (int d = 1; d < TPR; d *= 2) v[k] += __shfl_xor(v[k], d, kWave);
    }
  }
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

}  // namespace nf4moe
