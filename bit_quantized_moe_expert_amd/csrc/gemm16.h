// The bf16 matrix product that the dense operators are built on: a workgroup's tile of
//   acc[m][n] = sum_k X(m, k) Y(n, k),   fp32,
// for operands stored either way round, any sizes, K split as the caller likes.
//
// A tile is BM x BN with K in steps of 64, double buffered in LDS. A wave holds MB x NB
// blocks of v_mfma_f32_32x32x16_bf16. The n side is the instruction's first operand, so a
// lane's 16 values of a block lie in one row m = lane % 32 at n = 8 (i / 4) + 4 (lane / 32) +
// i % 4: a row's maximum or sum needs one exchange, with lane ^ 32, a row's own values
// (label, sum) are one register a block, and four neighbours in n are packed and stored
// together.
//
// Pipeline: a step's tile crosses memory -> registers -> LDS one step ahead of its use (the
// loads of step s + 2 are issued when those of s + 1 are written to LDS), fragments LDS ->
// registers one 16-deep slice ahead. The one barrier of a step comes before its last slice's
// products, so that the next step's first fragments load while these run.
//
// LDS layouts, without bank conflicts for the writes (16 bytes a lane, in order) and the
// fragment reads:
//  - an operand with k contiguous: rows of 64 k, 8 pieces of 16 bytes, piece c of row r at
//    place c ^ (r % 8); a fragment is one 16-byte read;
//  - an operand with its rows contiguous ("turned"): 64 rows of k, read by the transposing
//    ds_read_b64_tr_b16, which gives a lane four k of one column; 32-byte pieces stand at
//    p ^ (k % 4), so that the four k rows of a read lie in different banks.
#pragma once
#include "common.h"

namespace nf4moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGemmBK = 64;

// Loads through a buffer descriptor over 2^31 bytes from an address: an offset of kOutside
// is past its end and reads as zeros.
constexpr uint32_t kOutside = 0x80000000u;
__device__ inline __amdgpu_buffer_rsrc_t rsrc_at(const void *p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)kOutside, 0x00027000);
}
__device__ inline uint4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// One side of a tile: BR rows (of m or n) by a step's 64 k, on its way from memory to
// fragments.
template <int BR_, int THREADS, bool TURNED_>
struct GemmSide {
  static constexpr int BR = BR_;
  static constexpr bool TURNED = TURNED_;
  static constexpr int BYTES = BR * kGemmBK * 2;
  static constexpr int ROWC = TURNED ? BR / 8 : 8;                // pieces of an LDS row
  static constexpr int RSTEP = THREADS / ROWC;                    // LDS rows between a thread's pieces
  static constexpr int ROWS = TURNED ? kGemmBK : BR;              // LDS rows
  static constexpr int PER = ROWS >= RSTEP ? ROWS / RSTEP : 1;
  static_assert(THREADS % ROWC == 0 && (ROWS % RSTEP == 0 || ROWS < RSTEP), "pieces of a step");
  static_assert(!TURNED || BR >= 64, "the places of a turned row's pieces");

  const char *base[2];   // the tile's first element (pairs: of either array)
  int64_t kstep;         // bytes from a step to the next
  uint32_t voff[PER];
  uint4 regs[PER];
  int piece, row;        // this thread's piece of an LDS row, and its first row

  // Element (r, k) at p[r * ld + k], turned at p[k * ld + r]; the tile's first row is r0, rows at
  // or past `rows` read as zeros. ld and (turned) rows are multiples of 8, p is 16-byte
  // aligned, so a piece is wholly inside or left out; 256 rows of ld (turned: 64) are below 2^31 bytes.
  __device__ void init(const uint16_t *p, int64_t ld, int64_t r0, int64_t rows) {
    piece = threadIdx.x % ROWC, row = threadIdx.x / ROWC;
    if constexpr (TURNED) {
      base[0] = base[1] = reinterpret_cast<const char *>(p + r0);
      kstep = (int64_t)kGemmBK * ld * 2;
    } else {
      base[0] = base[1] = reinterpret_cast<const char *>(p + r0 * ld);
      kstep = kGemmBK * 2;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * RSTEP;
      const bool in = TURNED ? r0 + 8 * piece < rows && r < ROWS : r0 + r < rows && r < ROWS;
      voff[i] = in ? (uint32_t)(r * ld * 2 + piece * 16) : kOutside;
    }
  }
  // Pairs: of every 64 G rows of the tile the first 32 G are rows of one array (gate), the
  // others the same rows of another (up): p and q, `rows` each with one stride, r0 the first of
  // both. A thread's piece is of one array whatever the thread.
  template <int G>
  __device__ void init_pair(const uint16_t *p, const uint16_t *q, int64_t ld, int64_t r0, int64_t rows) {
    static_assert(!TURNED && RSTEP <= 32 * G && (32 * G) % RSTEP == 0, "a thread's piece is of one array");
    piece = threadIdx.x % ROWC, row = threadIdx.x / ROWC;
    base[0] = reinterpret_cast<const char *>(p + r0 * ld);
    base[1] = reinterpret_cast<const char *>(q + r0 * ld);
    kstep = kGemmBK * 2;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * RSTEP, at = r / (64 * G) * (32 * G) + r % (32 * G);
      voff[i] = r0 + at < rows ? (uint32_t)(at * ld * 2 + piece * 16) : kOutside;
    }
  }

  // The tile's part of k0 .. k0 + 63 to registers, zeros from kend on. live: bit k of the
  // step says whether its k row counts (turned sides with MASK).
  template <bool MASK, int G>
  __device__ void load(int64_t step, int left, uint64_t live) {
    const __amdgpu_buffer_rsrc_t r0 = rsrc_at(base[0] + step * kstep);
    const __amdgpu_buffer_rsrc_t r1 = rsrc_at(base[1] + step * kstep);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int k = TURNED ? row + i * RSTEP : piece * 8;
      bool in = k < left;
      if constexpr (MASK) in = in && (live >> (k & 63) & 1);
      const bool second = G > 0 && (i * RSTEP) / (32 * (G > 0 ? G : 1)) % 2;
      regs[i] = buffer_load16(second ? r1 : r0, in ? voff[i] : kOutside);
    }
  }
  __device__ void store(char *lds) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * RSTEP;
      if (ROWS < RSTEP && r >= ROWS) continue;
      const int at = TURNED ? piece ^ ((r & 3) << 1) : piece ^ (r & 7);
      *reinterpret_cast<uint4 *>(lds + (r * ROWC + at) * 16) = regs[i];
    }
  }
  // Fragment of the tile's rows 32 blk .. + 31 at k = 16 kk .. + 15: lane's row lane % 32, its k
  // 8 (lane / 32) .. + 7.
  __device__ static bf16x8_t frag(const char *lds, int blk, int kk) {
    const int lane = threadIdx.x & 63;
    if constexpr (!TURNED) {
      const int l32 = lane & 31, g = lane >> 5;
      return *reinterpret_cast<const bf16x8_t *>(lds + (blk * 32 + l32) * 128 + (((2 * kk + g) ^ (l32 & 7)) << 4));
    } else {
      const int i = lane & 15, half = lane >> 4 & 1, g = lane >> 5, kr = i >> 2;
      const int c = (((blk << 2) | (half << 1) | (i >> 1 & 1)) ^ (kr << 1));
      const char *at = lds + (kk * 16 + g * 8 + kr) * (ROWC * 16) + c * 16 + (i & 1) * 8;
      typedef __attribute__((address_space(3))) s16x4_t *lp;
      const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at));
      const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 4 * ROWC * 16));
      union {
        s16x4_t h[2];
        bf16x8_t v;
      } u;
      u.h[0] = a, u.h[1] = b;
      return u.v;
    }
  }
};

// MB x NB blocks of 32 x 32 a wave, WM x WN waves; XT / YT: a side is turned. G > 0: the n side
// is pairs (init_pair<G>). MASK: k rows of the turned n side count by their bit in `live`.
template <int MB_, int NB_, int WM_, int WN_, bool XT_ = false, bool YT_ = false, int G_ = 0, bool MASK_ = false>
struct GemmTile {
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, G = G_;
  static constexpr bool MASK = MASK_;
  static constexpr int BM = 32 * MB * WM, BN = 32 * NB * WN, THREADS = 64 * WM * WN;
  using X = GemmSide<BM, THREADS, XT_>;
  using Y = GemmSide<BN, THREADS, YT_>;
  static constexpr int STAGE = X::BYTES + Y::BYTES;
  // a row of a bf16 output tile in LDS, 16 bytes apart so that 16 rows lie in different banks
  static constexpr int PITCH = BN * 2 + 16;
  static constexpr int LDS = 2 * STAGE > BM * PITCH ? 2 * STAGE : BM * PITCH;
  X x;
  Y y;
  f32x16_t acc[NB][MB];

  // k values of [kbeg, kend), kbeg a multiple of 64 (0 without a split). live: a word for each 64 k.
  __device__ __attribute__((always_inline)) void run(char *lds, int64_t kbeg, int64_t kend, const uint64_t *live) {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[n][m][i] = 0.0f;
    const int64_t s0 = kbeg / kGemmBK, s1 = (kend + kGemmBK - 1) / kGemmBK;
    auto load = [&](int64_t s) __attribute__((always_inline)) {
      const int64_t l = kend - s * kGemmBK;
      const int left = (int)(l < kGemmBK ? l : kGemmBK);
      const uint64_t mask = MASK ? live[s] : 0;
      x.template load<false, 0>(s, left, 0);
      y.template load<MASK, G>(s, left, mask);
    };
    auto store = [&](int b) __attribute__((always_inline)) {
      x.store(lds + b * STAGE);
      y.store(lds + b * STAGE + X::BYTES);
    };
    bf16x8_t fx[2][MB], fy[2][NB];
    auto frags = [&](int b, int kk, int to) __attribute__((always_inline)) {
      const char *lx = lds + b * STAGE, *ly = lx + X::BYTES;
#pragma unroll
      for (int m = 0; m < MB; ++m) fx[to][m] = X::frag(lx, wm * MB + m, kk);
#pragma unroll
      for (int n = 0; n < NB; ++n) fy[to][n] = Y::frag(ly, wn * NB + n, kk);
    };
    auto mma = [&](int from) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m)
          acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy[from][n], fx[from][m], acc[n][m], 0, 0, 0);
    };
    if (s0 >= s1) return;
    load(s0);
    store(0);
    if (s0 + 1 < s1) load(s0 + 1);
    lds_barrier();
    frags(0, 0, 0);
    int b = 0;
    for (int64_t s = s0; s < s1; ++s, b ^= 1) {
      frags(b, 1, 1);
      mma(0);
      frags(b, 2, 0);
      if (s + 1 < s1) store(b ^ 1);
      mma(1);
      frags(b, 3, 1);
      if (s + 2 < s1) load(s + 2);
      mma(0);
      lds_barrier();
      if (s + 1 < s1) frags(b ^ 1, 0, 0);
      mma(1);
    }
    lds_barrier();  // the caller may use the LDS
  }
  __device__ static int wave_m() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) % WM; }
  __device__ static int wave_n() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) / WM; }
  // Tile row of this lane's values in block mb, and the first tile column of its group of four q in block nb.
  __device__ static int row_of(int mb) { return (wave_m() * MB + mb) * 32 + (int)(threadIdx.x & 31); }
  __device__ static int col_of(int nb, int q) {
    return (wave_n() * NB + nb) * 32 + 8 * q + 4 * (int)(threadIdx.x >> 5 & 1);
  }
};

// Rows of a bf16 tile in LDS (pitch bytes apart) to memory, 16 bytes a thread: COLS columns from
// byte `at` of a row on. rows and cols: how many exist (cols a multiple of 8, out 16-byte aligned).
template <int ROWS, int COLS, int THREADS>
__device__ inline void store_tile(const char *lds, int pitch, uint16_t *out, int64_t ld, int64_t rows, int64_t cols) {
  constexpr int C = COLS / 8, STEP = THREADS / C;
  static_assert(THREADS % C == 0 && ROWS % STEP == 0, "pieces of a tile");
  const int c = threadIdx.x % C, r0 = threadIdx.x / C;
  if (8 * c >= cols) return;
#pragma unroll
  for (int i = 0; i < ROWS / STEP; ++i) {
    const int r = r0 + i * STEP;
    if (r < rows) *reinterpret_cast<uint4 *>(out + r * ld + 8 * c) = *reinterpret_cast<const uint4 *>(lds + r * pitch + 16 * c);
  }
}
__device__ inline uint2 pack4(float a, float b, float c, float d) {
  return make_uint2(f32x2_to_bf16x2_rne(a, b), f32x2_to_bf16x2_rne(c, d));
}

// The tile of workgroup b of `total` = mt * nt: each XCD (b % 8) takes a run of tiles in an order
// that goes down 8 tiles of m, then on in n, so that the tiles it works on at a time share
// their operands in its L2. False where the workgroup has none.
__device__ inline bool gemm_tile_of(int b, int mt, int nt, int &m, int &n) {
  const int total = mt * nt, per = (total + 7) >> 3;
  const int at = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || at >= total) return false;
  const int band = at / (8 * nt), in = at - band * 8 * nt;
  const int high = mt - band * 8 < 8 ? mt - band * 8 : 8;
  m = band * 8 + in % high, n = in / high;
  return true;
}
inline int gemm_grid(int64_t mt, int64_t nt) { return (int)((mt * nt + 7) / 8 * 8); }

}  // namespace nf4moe
