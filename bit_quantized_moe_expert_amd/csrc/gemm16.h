// The bf16 matrix product that the dense operators are built on: a workgroup's tile of
//   acc[m][n] = sum_k X(m, k) Y(n, k),   fp32,
// for operands stored either way round, any sizes, K split as the caller likes.
//
// A tile is BM x BN with K in steps of 64. A wave holds MB x NB blocks of
// v_mfma_f32_16x16x32_bf16: under the card's power limit 2.06 PFLOP/s of random operands in
// registers, 1.82 with 32x32x16. The n side is the instruction's first operand, so a lane's
// four values of a block lie in one row m = lane % 16 at n = 4 (lane / 16) + i: a row's maximum
// or sum takes two exchanges, a row's own values (label, sum) are one register a block, and four
// neighbours in n are packed and stored together.
//
// Pipeline: buffer loads write LDS directly (16 bytes a lane, a wave's kilobyte in lane order); a
// step has four phases, 32 k by half of the wave's n blocks, and fragments go LDS -> registers
// one phase ahead. The one barrier of a step stands before its last phase: its own tile is then
// in registers, the next step's has landed, and the loads of the step after that go out into
// the place that is free now, in the last phase and the first of the next step. Loads and
// fragment reads are dealt out between the products.
//
// LDS layouts, without bank conflicts (64 banks, 256 bytes a cycle: 16 lanes of a 16-byte read, 32
// of an 8-byte one) for the fragment reads. A load's LDS places are fixed, so its lanes ask for
// the pieces (of 16 bytes) that belong there:
//  - an operand with k contiguous: rows of 64 k, 8 pieces, piece c of row r at place c ^ (r / 2 % 8),
//    two rows to the 256 bytes; a fragment is one 16-byte read. (Steps of 32 k, half a cache line
//    of each row at a time, ran 8 % below.)
//  - an operand with its rows contiguous ("turned"): 64 rows of k, read by the transposing
//    ds_read_b64_tr_b16, which gives a lane four k of one column; the eight k rows that 32
//    lanes take stand in different 32-byte pieces of the 256.
#pragma once
#include "common.h"

namespace nf4moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGemmBK = 64;

// A buffer descriptor over 2^31 bytes from an address: an offset of kOutside is past its end and
// reads as zeros.
constexpr uint32_t kOutside = 0x80000000u;
__device__ inline u32x4_t rsrc_at(const char *p) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, kOutside, 0x00027000u};
}
// 16 bytes a lane from the descriptor's memory to LDS at `lds` + 16 lane. The load has no output
// register; wait_loads and a barrier come before anyone reads what it wrote. (The compiler sets m0
// right before its own uses of it and keeps nothing there.)
__device__ inline void load_to_lds(u32x4_t rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(rsrc));
}
// Until at most N of this wave's loads (in order) are on their way.
template <int N>
__device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One side of a tile: BR rows (of m or n) by a step's 64 k, on its way from memory to fragments.
template <int BR_, int THREADS, bool TURNED_>
struct GemmSide {
  static constexpr int BR = BR_;
  static constexpr bool TURNED = TURNED_;
  static constexpr int BYTES = BR * kGemmBK * 2;
  static constexpr int ROWC = TURNED ? BR / 8 : kGemmBK / 8;      // pieces of an LDS row
  static constexpr int ROWS = TURNED ? kGemmBK : BR;              // LDS rows
  static constexpr int RSTEP = THREADS / ROWC;                    // LDS rows between a thread's pieces
  static constexpr int PER = ROWS / RSTEP;
  static_assert(THREADS % ROWC == 0 && ROWS % RSTEP == 0 && PER > 0, "pieces of a step");
  static_assert(RSTEP % 16 == 0, "a thread's pieces have one place in their rows");
  static_assert(!TURNED || BR >= 64, "the places of a turned row's pieces");

  const char *base[2];   // the tile's first element (pairs: of either array)
  int64_t kstep;         // bytes from a step to the next
  uint32_t voff[PER];
  int piece, row;        // this thread's piece of an LDS row, and its first row

  // Where the pieces of k row k of a turned side stand.
  __device__ static int turned_swizzle(int k) {
    return ROWC >= 16 ? (k & 3) << 1 | (k & 8) : (k & 2) | (k & 8) >> 1;
  }
  __device__ void place() {
    row = threadIdx.x / ROWC;
    piece = (int)(threadIdx.x % ROWC) ^ (TURNED ? turned_swizzle(row) : row >> 1 & 7);
  }

  // Element (r, k) at p[r * ld + k], turned at p[k * ld + r]; the tile's first row is r0, rows at
  // or past `rows` read as zeros. ld and (turned) rows are multiples of 8, p is 16-byte
  // aligned, so a piece is wholly inside or left out; 256 rows of ld (turned: 64) are below 2^31 bytes.
  __device__ void init(const uint16_t *p, int64_t ld, int64_t r0, int64_t rows) {
    place();
    base[0] = base[1] = reinterpret_cast<const char *>(p + (TURNED ? r0 : r0 * ld));
    kstep = kGemmBK * 2 * (TURNED ? ld : 1);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * RSTEP;
      const bool in = TURNED ? r0 + 8 * piece < rows : r0 + r < rows;
      voff[i] = in ? (uint32_t)(r * ld * 2 + piece * 16) : kOutside;
    }
  }
  // Pairs: of every 32 G rows of the tile the first 16 G are rows of one array (gate), the
  // others the same rows of another (up): p and q, `rows` each with one stride, r0 the first of
  // both. A thread's piece is of one array whatever the thread.
  template <int G>
  __device__ void init_pair(const uint16_t *p, const uint16_t *q, int64_t ld, int64_t r0, int64_t rows) {
    static_assert(!TURNED && 16 * G % RSTEP == 0, "a thread's piece is of one array");
    place();
    base[0] = reinterpret_cast<const char *>(p + r0 * ld);
    base[1] = reinterpret_cast<const char *>(q + r0 * ld);
    kstep = kGemmBK * 2;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * RSTEP, at = r / (32 * G) * (16 * G) + r % (16 * G);
      voff[i] = r0 + at < rows ? (uint32_t)(at * ld * 2 + piece * 16) : kOutside;
    }
  }

  // Piece i of a step's 64 k to LDS at `lds` (this side's stage), zeros from `left` on. live: bit k
  // says whether the step's k row counts (turned sides with MASK).
  template <bool MASK, int G>
  __device__ void load(int i, int64_t step, int left, uint64_t live, uint32_t lds) const {
    const int k = TURNED ? row + i * RSTEP : piece * 8;
    bool in = k < left;
    if constexpr (MASK) in = in && (live >> (k & 63) & 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int which = G > 0 ? i * RSTEP / (16 * (G > 0 ? G : 1)) % 2 : 0;
    load_to_lds(rsrc_at(base[which] + step * kstep), in ? voff[i] : kOutside,
                lds + (uint32_t)(wave * 64 + i * THREADS) * 16);
  }
  // Fragment of the tile's rows 16 blk .. + 15 at the step's k 32 kk .. + 31: lane's row lane % 16, its k
  // 8 (lane / 16) .. + 7.
  __device__ static bf16x8_t frag(const char *lds, int blk, int kk) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    if constexpr (!TURNED) {
      return *reinterpret_cast<const bf16x8_t *>(lds + (blk * 16 + i) * 128 + (((4 * kk + g) ^ (i >> 1)) << 4));
    } else {
      const int k = kk * 32 + g * 8 + (i >> 2);
      const int c = ((blk << 1) | (i >> 1 & 1)) ^ turned_swizzle(k);
      const char *at = lds + k * (ROWC * 16) + c * 16 + (i & 1) * 8;
      typedef __attribute__((address_space(3))) s16x4_t *lp;
      union {
        s16x4_t h[2];
        bf16x8_t v;
      } u;
      u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at));
      u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 4 * ROWC * 16));   // (k + 4: the same places)
      return u.v;
    }
  }
};

// MB x NB blocks of 16 x 16 a wave, WM x WN waves; XT / YT: a side is turned. G > 0: the n side
// is pairs (init_pair<G>). MASK: k rows of the turned n side count by their bit in `live`.
template <int MB_, int NB_, int WM_, int WN_, bool XT_ = false, bool YT_ = false, int G_ = 0, bool MASK_ = false>
struct GemmTile {
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, G = G_;
  static constexpr bool MASK = MASK_;
  static constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN, THREADS = 64 * WM * WN;
  static_assert(NB % 2 == 0, "two halves of the n blocks");
  using X = GemmSide<BM, THREADS, XT_>;
  using Y = GemmSide<BN, THREADS, YT_>;
  // Steps of either side in LDS (a third of x, 160 KB, gained nothing).
  static constexpr int XS = 2, YS = 2, YAT = XS * X::BYTES;
  static_assert(YS == 2 && XS >= YS, "the order of the loads");
  // a row of a bf16 output tile in LDS, 16 bytes apart so that 16 rows lie in different banks
  static constexpr int PITCH = BN * 2 + 16;
  static constexpr int STAGES = YAT + YS * Y::BYTES, LDS = STAGES > BM * PITCH ? STAGES : BM * PITCH;
  X x;
  Y y;
  f32x4_t acc[NB][MB];

  // k values of [kbeg, kend), kbeg a multiple of 64 (0 without a split). live: a word for each 64 k.
  __device__ __attribute__((always_inline)) void run(char *lds, int64_t kbeg, int64_t kend, const uint64_t *live) {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        acc[n][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t s0 = kbeg / kGemmBK, s1 = (kend + kGemmBK - 1) / kGemmBK;
    if (s0 >= s1) return;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    constexpr int P = X::PER + Y::PER, NP = NB / 2;
    // Piece i (first of y, then of x) of the steps whose turn it is; past the end zeros, so that the
    // number of loads on their way is known.
    auto left = [&](int64_t s) __attribute__((always_inline)) {
      const int64_t l = kend - s * kGemmBK;
      return (int)(l < kGemmBK ? l : kGemmBK);
    };
    auto load_x = [&](int64_t s, int i) __attribute__((always_inline)) {
      x.template load<false, 0>(i, s, left(s), 0, lds0 + (uint32_t)((s - s0) % XS) * X::BYTES);
    };
    auto load_y = [&](int64_t s, int i) __attribute__((always_inline)) {
      y.template load<MASK, G>(i, s, left(s), MASK && s < s1 ? live[s] : 0, lds0 + YAT + (uint32_t)((s - s0) % YS) * Y::BYTES);
    };
    auto load = [&](int64_t done, int i) __attribute__((always_inline)) {   // where step `done` was
      if (i < Y::PER) load_y(done + YS, i);
      else if (i < P) load_x(done + XS, i - Y::PER);
    };
    bf16x8_t fx[2][MB], fy[2][NP];
    // Phase p: k slice p / 2, half p % 2 of the n blocks.
    auto frag_y = [&](int64_t s, int p, int n) __attribute__((always_inline)) {
      fy[p & 1][n] = Y::frag(lds + YAT + (int)((s - s0) % YS) * Y::BYTES, wn * NB + p % 2 * NP + n, p / 2);
    };
    auto frag_x = [&](int64_t s, int p, int m) __attribute__((always_inline)) {
      fx[p / 2][m] = X::frag(lds + (int)((s - s0) % XS) * X::BYTES, wm * MB + m, p / 2);
    };
    auto mma = [&](int p, int n) __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        f32x4_t &c = acc[p % 2 * NP + n][m];
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fy[p & 1][n], fx[p / 2][m], c, 0, 0, 0);
      }
    };
    constexpr int P3 = P / 2;   // loads in the last phase, the others in the next step's first
#pragma unroll
    for (int j = -XS; j < 0; ++j)
#pragma unroll
      for (int i = 0; i < (j == -1 ? P3 : P); ++i)
        if (j + (i < Y::PER ? YS : XS) >= 0) load(s0 + j, i);
    wait_loads<(XS - 2) * X::PER + P3>();
    lds_barrier();
#pragma unroll
    for (int n = 0; n < NP; ++n) frag_y(s0, 0, n);
#pragma unroll
    for (int m = 0; m < MB; ++m) frag_x(s0, 0, m);
    for (int64_t s = s0; s < s1; ++s) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (p == 3) {
          wait_loads<(XS - 2) * X::PER>();   // step s + 1 has landed
          lds_barrier();
        }
        const int64_t of = p == 3 ? s + 1 : s;
        const int q = (p + 1) % 4;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          frag_y(of, q, n);
          if (q % 2 == 0) {
#pragma unroll
            for (int m = n * MB / NP; m < (n + 1) * MB / NP; ++m) frag_x(of, q, m);
          }
          if (p == 3) {
#pragma unroll
            for (int i = n * P3 / NP; i < (n + 1) * P3 / NP; ++i) load(s, i);
          }
          if (p == 0) {
#pragma unroll
            for (int i = P3 + n * (P - P3) / NP; i < P3 + (n + 1) * (P - P3) / NP; ++i) load(s - 1, i);
          }
          mma(p, n);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    wait_loads<0>();
    lds_barrier();  // the caller may use the LDS
  }
  __device__ static int wave_m() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) % WM; }
  __device__ static int wave_n() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) / WM; }
  // Tile row of this lane's values in block mb, and the first tile column of its four in block nb.
  __device__ static int row_of(int mb) { return (wave_m() * MB + mb) * 16 + (int)(threadIdx.x & 15); }
  __device__ static int col_of(int nb) { return (wave_n() * NB + nb) * 16 + 4 * (int)(threadIdx.x >> 4 & 3); }
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
// that goes down 4 tiles of m, then on in n, so that the tiles it works on at a time share
// their operands in its L2. False where the workgroup has none.
__device__ inline bool gemm_tile_of(int b, int mt, int nt, int &m, int &n) {
  const int total = mt * nt, per = (total + 7) >> 3;
  const int at = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || at >= total) return false;
  const int band = at / (4 * nt), in = at - band * 4 * nt;
  const int high = mt - band * 4 < 4 ? mt - band * 4 : 4;
  m = band * 4 + in % high, n = in / high;
  return true;
}
inline int gemm_grid(int64_t mt, int64_t nt) { return (int)((mt * nt + 7) / 8 * 8); }

}  // namespace nf4moe
