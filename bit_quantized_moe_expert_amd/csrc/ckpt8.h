// The 8-bit checkpoint formats (device side) and 8-element loads and stores
// shared by the training kernels.
//
// Both formats are OCP MX v1.0 element types over blocks of 32 consecutive
// elements with one e8m0 scale byte b (multiplier 2^(b - 127)):
//   0 MXINT8      X = floor(log2 amax), code = RNE(v / 2^(X - 6)) in [-127, 127]
//   1 MXFP8 e4m3  X = floor(log2 amax) - 8, code = e4m3 RNE(v / 2^X), saturated at 448
// with X clamped to at least -127 and b = X + 127. The scale is a power of two,
// so v / 2^X is exact and a code is a function of the input alone: nothing
// depends on how a division was rounded. A decoded value has at most 7
// significant bits, so it is exact in bf16 (down to bf16's own subnormals). A
// block with a NaN or an infinity has b = 255 and decodes to NaN as a whole.
#pragma once
#include "common.h"

namespace nf4moe {

enum Ckpt8Fmt { CK_NONE = -1, CK_MXINT8 = 0, CK_MXFP8 = 1 };

// 16 bytes at an address of any alignment (the hardware's unaligned access
// mode, on by default, takes one instruction whatever the address).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
__device__ inline uint4 load16(const void *p) {
  const u32x4_any v = *reinterpret_cast<const u32x4_any *>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ inline void store16(void *p, uint4 v) {
  u32x4_any u = {v.x, v.y, v.z, v.w};
  *reinterpret_cast<u32x4_any *>(p) = u;
}
// ... past the caches, for long arrays that are read or written once.
__device__ inline void store16_nt(void *p, uint4 v) {
  u32x4_any u = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any *>(p));
}
__device__ inline uint4 load16_nt(const void *p) {
  const u32x4_any v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ inline uint2 load8(const void *p) {
  const u32x2_any v = *reinterpret_cast<const u32x2_any *>(p);
  return make_uint2(v.x, v.y);
}
typedef uint32_t u32_any __attribute__((aligned(1)));
__device__ inline void store4(void *p, uint32_t v) { *reinterpret_cast<u32_any *>(p) = v; }
__device__ inline void store8(void *p, uint2 v) {
  u32x2_any u = {v.x, v.y};
  *reinterpret_cast<u32x2_any *>(p) = u;
}

__device__ inline void unpack_bf16x8(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo_to_f32(u[i]);
    v[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}
__device__ inline uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]),
                    f32x2_to_bf16x2_rne(v[4], v[5]), f32x2_to_bf16x2_rne(v[6], v[7]));
}

// Eight consecutive elements at index i of a bf16 (BF = true) or fp32 array.
template <bool BF, bool NT = false>
__device__ inline void load_elems8(const void *p, int64_t i, float (&v)[8]) {
  if constexpr (BF) {
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p) + i;
    unpack_bf16x8(NT ? load16_nt(h) : load16(h), v);
  } else {
    const float *f = reinterpret_cast<const float *>(p) + i;
    const uint4 a = NT ? load16_nt(f) : load16(f), b = NT ? load16_nt(f + 4) : load16(f + 4);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  }
}
template <bool BF>
__device__ inline void store_elems8(void *p, int64_t i, const float (&v)[8]) {
  if constexpr (BF) {
    store16(reinterpret_cast<uint16_t *>(p) + i, pack_bf16x8(v));
  } else {
    float *f = reinterpret_cast<float *>(p) + i;
    store16(f, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    store16(f + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  }
}

// Largest magnitude as bits (ordered like the value; a NaN is above infinity).
__device__ inline uint32_t abs_bits_max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    m = a > m ? a : m;
  }
  return m;
}
// ... over aligned groups of 2 or 4 lanes.
template <int LANES>
__device__ inline uint32_t lanes_max_u32(uint32_t m) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false);  // quad_perm [1,0,3,2]
  m = o > m ? o : m;
  if (LANES == 4) {
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false);         // quad_perm [2,3,0,1]
    m = o > m ? o : m;
  }
  return m;
}

// Scale byte of a block whose largest magnitude has these bits. A subnormal
// maximum has exponent field 0, i.e. X = -127, the clamp.
template <int FMT>
__device__ inline uint32_t ckpt8_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  if (e == 255) return 255u;
  return (uint32_t)(FMT == CK_MXINT8 ? e : (e > 8 ? e - 8 : 0));
}

// Codes of 8 elements under scale byte b, four to a word, first element lowest.
template <int FMT>
__device__ inline uint2 ckpt8_encode8(const float (&v)[8], uint32_t b) {
  if (b == 255u) return make_uint2(0u, 0u);
  uint32_t w[2];
  if constexpr (FMT == CK_MXINT8) {
    const int sh = 133 - (int)b;  // v / 2^(b - 127 - 6), by the exponent: exact
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[4 * h + i], sh), -127.0f, 127.0f);
        c[i] = __float_as_uint(t + 12582912.0f);  // + 1.5 * 2^23: the low byte is RNE(t) in two's complement
      }
      const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
      w[h] = lo | hi;
    }
  } else {
    const int sh = 127 - (int)b;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        t[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[4 * h + i], sh), -448.0f, 448.0f);
      int r = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);  // OCP e4m3, RNE
      r = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], r, true);
      w[h] = (uint32_t)r;
    }
  }
  return make_uint2(w[0], w[1]);
}

// The multiplier of a code's own value (an integer, or an e4m3 number).
template <int FMT>
__device__ inline float ckpt8_multiplier(uint32_t b) {
  if (b == 255u) return __builtin_nanf("");
  if constexpr (FMT == CK_MXINT8)  // 2^(b - 133), subnormal for b <= 6
    return __uint_as_float(b > 6u ? (b - 6u) << 23 : 1u << (b + 16u));
  else
    return __uint_as_float(b > 0u ? b << 23 : 0x400000u);
}

template <int FMT>
__device__ inline void ckpt8_decode8(uint2 q, uint32_t b, float (&v)[8]) {
  const float m = ckpt8_multiplier<FMT>(b);
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == CK_MXINT8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = (float)(int8_t)(w[h] >> (8 * i)) * m;
    } else {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
      const auto c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
      v[4 * h] = a[0] * m, v[4 * h + 1] = a[1] * m, v[4 * h + 2] = c[0] * m, v[4 * h + 3] = c[1] * m;
    }
  }
}

}  // namespace nf4moe
