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
// fragment reads are dealt out between the products. A workgroup goes through several tiles
// without draining this: the loads run on into the next tile's first steps while the tile's
// epilogue works, in a part of LDS of its own, a wave for itself and without barriers.
//
// What bounds it is the card's power: the products alone, from registers, would take it to 2060
// TFLOP/s, with their operands on the way from LDS and memory it settles at 8192^3 at 1475 with both
// operands k contiguous, 1400 with one turned and 1365 with both (a library's product there, by
// the box: 1460 to 1632, 1360 to 1419, 1176 to 1223). So what saves instructions and LDS traffic
// pays, and idle CUs at the end of a launch cost less than their share: the others run faster.
// Ragged edges are whole tiles of zeros; wider waves (128 x 128 of four) do not fit the registers.
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
  const uint64_t a = (uint64_t)p;   // the same in every lane
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)), kOutside, 0x00027000u};
}
// 16 bytes a lane from the descriptor's memory to LDS at `lds` + 16 lane. The load has no output
// register; wait_loads and a barrier come before anyone reads what it wrote. (The compiler sets m0
// right before its own uses of it and keeps nothing there.)
__device__ inline void load_to_lds(u32x4_t rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane((int)lds)),
               "v"(off), "s"(rsrc));
}
// Until at most N of this wave's loads (in order) are on their way.
template <int N>
__device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Orders a wave's LDS accesses, whose lanes read what others wrote (the hardware keeps their order).
__device__ inline void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// k values of [kbeg, kend), kbeg a multiple of 64; at least one step (of zeros where there is none).
struct GemmRange {
  int64_t kbeg, kend;
  __device__ int64_t first() const { return kbeg / kGemmBK; }
  __device__ int64_t last() const {
    const int64_t l = (kend + kGemmBK - 1) / kGemmBK;
    return l > first() ? l : first() + 1;
  }
  // Part g of n, whole steps; the first is the longest.
  __device__ GemmRange part(int g, int n) const {
    const int64_t each = (last() - first() + n - 1) / n * kGemmBK, b = kbeg + g * each;
    return {b, b + each < kend ? b + each : kend};
  }
};

// One side of a tile: BR rows (of m or n) by a step's 64 k, on its way from memory to fragments, moved by
// THREADS threads (`tid` among them).
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
  __device__ static int tid() { return (int)threadIdx.x % THREADS; }
  __device__ static int wave() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) % (THREADS / 64); }
  __device__ void place() {
    row = tid() / ROWC;
    piece = tid() % ROWC ^ (TURNED ? turned_swizzle(row) : row >> 1 & 7);
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

  __device__ void no_more() {
#pragma unroll
    for (int i = 0; i < PER; ++i) voff[i] = kOutside;
  }

  // Piece i of a step's 64 k to LDS at `lds` (this side's stage), zeros from `left` on. live: bit k
  // says whether the step's k row counts (turned sides with MASK).
  template <bool MASK, int G>
  __device__ void load(int i, int64_t step, int left, uint64_t live, uint32_t lds) const {
    const int k = TURNED ? row + i * RSTEP : piece * 8;
    bool in = k < left;
    if constexpr (MASK) in = in && (live >> (k & 63) & 1);
    const int which = G > 0 ? i * RSTEP / (16 * (G > 0 ? G : 1)) % 2 : 0;
    load_to_lds(rsrc_at(base[which] + step * kstep), in ? voff[i] : kOutside,
                lds + (uint32_t)(wave() * 64 + i * THREADS) * 16);
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
// is pairs (init_pair<G>). MASK: k rows of the turned n side count by their bit in `live`. KS > 1: so many
// groups of WM x WN waves share a tile, each with a part of its k (small products, whose time is the
// steps' latency); a workgroup has one tile then.
template <int MB_, int NB_, int WM_, int WN_, bool XT_ = false, bool YT_ = false, int G_ = 0, bool MASK_ = false, int KS_ = 1>
struct GemmTile {
  static constexpr int KS = KS_, GROUP = 64 * WM_ * WN_;
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, G = G_;
  static constexpr bool MASK = MASK_;
  static constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN, THREADS = GROUP * KS;
  static_assert(NB % 2 == 0, "two halves of the n blocks");
  using X = GemmSide<BM, GROUP, XT_>;
  using Y = GemmSide<BN, GROUP, YT_>;
  // Two steps in LDS, and behind them for each wave a block row of its output in bf16.
  static constexpr int STAGE = X::BYTES + Y::BYTES, SCRATCH = 512 * NB, LDS = 2 * STAGE * KS + SCRATCH * WM * WN;
  // workgroups that run at a time (by LDS, and 16 waves a CU at these kernels' registers)
  static constexpr int BY_LDS = (160 << 10) / LDS, BY_WAVES = 16 / (WM * WN * KS);
  static constexpr int PER_CU = BY_LDS < BY_WAVES ? BY_LDS : BY_WAVES, MOST = 256 * PER_CU;
  static constexpr int WAVES_SIMD = (PER_CU * WM * WN * KS + 3) / 4;
  X x;
  Y y;
  f32x4_t acc[NB][MB];

  // All of the workgroup's tiles. place(r, x, y): the sides of tile r and its k range (false: there is no
  // tile r; tile 0 exists); done(r): the epilogue, with the sums in acc. live: a word for each 64 k.
  template <class Place, class Done>
  __device__ __attribute__((always_inline)) void run(char *lds, const uint64_t *live, Place place, Done done) {
    const int wm = wave_m(), wn = wave_n(), group = KS > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / GROUP) : 0;
    char *const all = lds;
    if constexpr (KS > 1) lds += group * 2 * STAGE;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    constexpr int P = X::PER + Y::PER, NP = NB / 2, P3 = P / 2;   // P3 loads in a step's last phase, the others in the next one's first
    // where the loads are: tile, step, and what they may touch
    int tile = 0;
    GemmRange at;
    uint64_t mask = 0;
    place(0, x, y, at);
    if constexpr (KS > 1) at = at.part(group, KS);
    int64_t step = at.first();
    auto read_mask = [&]() __attribute__((always_inline)) {
      if constexpr (MASK) mask = step * kGemmBK < at.kend ? live[step] : 0;
    };
    auto load = [&](int stage, int i) __attribute__((always_inline)) {
      const int64_t l = at.kend - step * kGemmBK;
      const int left = (int)(l < kGemmBK ? l : kGemmBK);
      const uint32_t to = lds0 + (uint32_t)stage * STAGE;
      if (i < Y::PER) y.template load<MASK, G>(i, step, left, mask, to + X::BYTES);
      else x.template load<false, 0>(i - Y::PER, step, left, 0, to);
    };
    auto advance = [&]() __attribute__((always_inline)) {
      if (++step < at.last()) return;
      if (KS == 1 && place(++tile, x, y, at)) {
        step = at.first();
      } else {
        x.no_more(), y.no_more();
        step = 0, at = {0, 0};
      }
    };
    bf16x8_t fx[2][MB], fy[2][NP];
    // Phase p: k slice p / 2, half p % 2 of the n blocks.
    auto frag_y = [&](int stage, int p, int n) __attribute__((always_inline)) {
      fy[p & 1][n] = Y::frag(lds + stage * STAGE + X::BYTES, wn * NB + p % 2 * NP + n, p / 2);
    };
    auto frag_x = [&](int stage, int p, int m) __attribute__((always_inline)) {
      fx[p / 2][m] = X::frag(lds + stage * STAGE, wm * MB + m, p / 2);
    };
    read_mask();
#pragma unroll
    for (int i = 0; i < P; ++i) load(0, i);
    advance();
    read_mask();
#pragma unroll
    for (int i = 0; i < P3; ++i) load(1, i);
    wait_loads<P3>();
    lds_barrier();
    int stage = 0;
    GemmRange now;
    for (int r = 0; (KS == 1 || r == 0) && place.range(r, now); ++r) {
      if constexpr (KS > 1) now = now.part(0, KS);   // as many steps for every group
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[n][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < NP; ++n) frag_y(stage, 0, n);   // (again: no registers are held through an epilogue)
#pragma unroll
      for (int m = 0; m < MB; ++m) frag_x(stage, 0, m);
      for (int64_t s = now.first(); s < now.last(); ++s, stage ^= 1) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p == 1) advance();
          if (p == 3) {
            wait_loads<0>();   // the next step has landed
            lds_barrier();
          }
          const int of = p == 3 ? stage ^ 1 : stage, q = (p + 1) % 4;
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            frag_y(of, q, n);
            if (q % 2 == 0) {
#pragma unroll
              for (int m = n * MB / NP; m < (n + 1) * MB / NP; ++m) frag_x(of, q, m);
            }
            if (p == 2 && n == 0) read_mask();   // its wait is the barrier's
            if (p == 3) {
#pragma unroll
              for (int i = n * P3 / NP; i < (n + 1) * P3 / NP; ++i) load(stage, i);
            }
            if (p == 0) {
#pragma unroll
              for (int i = P3 + n * (P - P3) / NP; i < P3 + (n + 1) * (P - P3) / NP; ++i) load(stage ^ 1, i);
            }
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              f32x4_t &c = acc[p % 2 * NP + n][m];
              c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fy[p & 1][n], fx[p / 2][m], c, 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if constexpr (KS > 1) {   // the groups' sums, added in their order
        wait_loads<0>();
        lds_barrier();
        const int t = X::tid();
        f32x4_t *mine = reinterpret_cast<f32x4_t *>(lds);
        static_assert(NB * MB * 16 * GROUP <= 2 * STAGE, "a group's sums in its own stages");
        if (group > 0) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MB; ++m) mine[(n * MB + m) * GROUP + t] = acc[n][m];
        }
        lds_barrier();
        if (group > 0) return;   // the wave; no barrier follows
        for (int g = 1; g < KS; ++g) {
          const f32x4_t *other = reinterpret_cast<const f32x4_t *>(all + g * 2 * STAGE);
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MB; ++m) acc[n][m] += other[(n * MB + m) * GROUP + t];
        }
      }
      done(r);
    }
    if constexpr (KS > 1) return;
    wait_loads<0>();   // none may land after the workgroup's LDS is another's
  }
  __device__ static int wave_m() { return X::wave() % WM; }
  __device__ static int wave_n() { return X::wave() / WM; }
  // First tile row of this wave's block row mb (a lane's values are of its row lane % 16), first tile
  // column of the wave, and the wave's column of a lane's four in block nb.
  __device__ static int row_at(int mb) { return (wave_m() * MB + mb) * 16; }
  __device__ static int cols_at() { return wave_n() * NB * 16; }
  __device__ static int col_of(int lane, int nb) { return nb * 16 + 4 * (lane >> 4); }
  __device__ static char *scratch(char *lds) {
    return lds + 2 * STAGE * KS + X::wave() * SCRATCH;
  }
};

// The lane, as a value that epilogues' addresses are computed from where they are needed and not
// before the main loop, whose registers they would take.
__device__ inline int epilogue_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}
__device__ inline uint2 pack4(float a, float b, float c, float d) {
  return make_uint2(f32x2_to_bf16x2_rne(a, b), f32x2_to_bf16x2_rne(c, d));
}
// What bf16 leaves of v, a value's second part: nothing where bf16 has it infinite (v finite or not) or NaN, so that
// the first part alone says so.
__device__ inline float bf16_rest(float v) {
  const float r = bf16_to_f32(f32_to_bf16_rne(v));
  return fabsf(r) < __builtin_inff() ? v - r : 0.0f;
}

// A wave's block row, 16 rows of COLS bf16, on its way from the products' layout to whole rows in
// memory: through the wave's own LDS, 16-byte pieces moved so that neither side has bank
// conflicts, and out in 16 bytes a lane.
template <int COLS>
struct BlockRow {
  static constexpr int C = COLS / 8;
  static_assert(C == 16 || C == 8 || C == 4 || C == 2, "pieces of a row");
  char *lds;
  int lane;
  __device__ static int place(int row, int piece) { return (row * C + (piece ^ (row * C / 16))) * 16; }
  // four values of this lane's row, from column `col` on (a multiple of 4)
  __device__ void put(int col, uint2 v) const {
    *reinterpret_cast<uint2 *>(lds + place(lane & 15, col >> 3) + (col & 4) * 2) = v;
  }
  __device__ uint16_t *one(int row, int col) const {
    return reinterpret_cast<uint16_t *>(lds + place(row, col >> 3) + (col & 7) * 2);
  }
  // rows and cols: how many exist (cols a multiple of 8, out 16-byte aligned)
  __device__ void out(uint16_t *to, int64_t ld, int64_t rows, int64_t cols) const {
    wave_lds_order();
    const int c = lane % C;
    constexpr int N = 16 * C / 64 > 0 ? 16 * C / 64 : 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = lane / C + i * (64 / C);
      if (r < rows && r < 16 && 8 * c < cols)
        *reinterpret_cast<uint4 *>(to + r * ld + 8 * c) = *reinterpret_cast<const uint4 *>(lds + place(r, c));
    }
    wave_lds_order();
  }
};

// Up to 16 rows of x against 16 rows of y, for few workgroups of them: W waves share K, each lane loads its
// fragments from memory as they are needed, eight steps at a time, and the waves' sums meet in LDS. A row of either side
// is any row: y_row(i) and x_row(i) for i in 0 .. 15 (rows that do not exist: any that do, their sums are not used).
template <int W>
struct FewRows {
  static constexpr int THREADS = 64 * W, LDS = W * 1024;
  // The sums in wave 0, as GemmTile's acc holds them.
  template <class YRow, class XRow>
  __device__ __attribute__((always_inline)) static f32x4_t run(char *lds, int K, YRow y_row, XRow x_row) {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const uint16_t *yp = y_row(i), *xp = x_row(i);
    f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int pieces = K / 8, steps = (pieces + 3) / 4, first = steps * wave / W, last = steps * (wave + 1) / W;
    constexpr int U = 8;   // steps in flight
    for (int s0 = first; s0 < last; s0 += U) {
      uint4 ry[U], rx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (s0 + u) * 4 + g, in = at < pieces ? at : 0;
        ry[u] = *reinterpret_cast<const uint4 *>(yp + 8 * in);
        rx[u] = *reinterpret_cast<const uint4 *>(xp + 8 * in);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = s0 + u < last && (s0 + u) * 4 + g < pieces;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, in ? ry[u] : zero),
                                                      __builtin_bit_cast(bf16x8_t, in ? rx[u] : zero), acc, 0, 0, 0);
      }
    }
    f32x4_t *red = reinterpret_cast<f32x4_t *>(lds);
    red[wave * 64 + lane] = acc;
    lds_barrier();
    f32x4_t sum = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) sum += red[w * 64 + lane];
    }
    return sum;
  }
};

// Up to 32 rows of x against 64 rows of y, many of them: a stream of y's steps of 64 k through a
// ring of STAGES places in LDS, all but two of them on their way (Y_GROUP: y's rows are pairs, as GemmTile's G). 17 rows against 32003 of
// 2048 k, statistics and loss with them: 31.8 us with six places (two workgroups a CU), 34.2 with four (three),
// 35.3 with eight (one), and 38.4 with loads to registers as in FewRows, whose next ones wait for their sums.
template <int STAGES, int Y_GROUP>
struct FewStream {
  static constexpr int THREADS = 256;
  using X = GemmSide<32, THREADS, false>;
  using Y = GemmSide<64, THREADS, false>;
  static constexpr int STAGE = X::BYTES + Y::BYTES, LDS = STAGES * STAGE, P = X::PER + Y::PER;
  // step(x, y): the products of a step of 64 k from its places (GemmSide's frag). The workgroup's LDS is free after it.
  template <class Step>
  __device__ __attribute__((always_inline)) static void run(char *lds, int K, const X &x, const Y &y, Step step) {
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const int steps = (K + kGemmBK - 1) / kGemmBK;
    auto load = [&](int s, int stage) __attribute__((always_inline)) {
      const int left = K - s * kGemmBK;   // (none past the end: zeros)
      const uint32_t to = lds0 + (uint32_t)stage * STAGE;
#pragma unroll
      for (int i = 0; i < Y::PER; ++i) y.template load<false, Y_GROUP>(i, s, left, 0, to + X::BYTES);
#pragma unroll
      for (int i = 0; i < X::PER; ++i) x.template load<false, 0>(i, s, left, 0, to);
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) load(s, s);
    int at = 0;
    for (int s = 0; s < steps; ++s) {
      wait_loads<P *(STAGES - 2)>();
      lds_barrier();   // step s has landed, and step s - 1's place has been read
      load(s + STAGES - 1, at == 0 ? STAGES - 1 : at - 1);
      step(lds + at * STAGE, lds + at * STAGE + X::BYTES);
      at = at + 1 == STAGES ? 0 : at + 1;
    }
    wait_loads<0>();
    lds_barrier();
  }
};

// The tiles of workgroup b of nb (a multiple of 8) of mt * nt tiles in `slices` of k: each XCD (b % 8)
// takes a run of tiles in an order that goes down 4 tiles of m, then on in n, so that the 32
// tiles that it works on at a time share their operands in its L2 (without this 1064 TFLOP/s for 1470).
struct GemmTiles {
  int b, nb, mt, nt, slices;
  int64_t K;
  int log = 3;   // of the XCDs that b counts through
  __device__ bool find(int r, int &m, int &n, int &slice) const {
    const int xcds = 1 << log, each = mt * nt, total = each * slices, per = (total + xcds - 1) >> log, i = (b >> log) + r * (nb >> log);
    const int at = (b & (xcds - 1)) * per + i;
    if (i >= per || at >= total) return false;
    slice = at / each;
    const int in = at - slice * each, band = in / (4 * nt), rest = in - band * 4 * nt;
    const int high = mt - band * 4 < 4 ? mt - band * 4 : 4;
    n = rest / high, m = band * 4 + rest - n * high;
    return true;
  }
  // slices of whole steps
  __device__ GemmRange range_of(int slice) const {
    const int64_t steps = (K + kGemmBK - 1) / kGemmBK, each = (steps + slices - 1) / slices, k0 = slice * each * kGemmBK;
    return {k0, k0 + each * kGemmBK < K ? k0 + each * kGemmBK : K};
  }
  __device__ bool range(int r, GemmRange &g) const {
    int m, n, slice;
    if (!find(r, m, n, slice)) return false;
    g = range_of(slice);
    return true;
  }
};
// About how long `tiles` tiles take that run `slots` at a time, in rounds of 256 tiles of 256 x 256: a
// whole round takes `full`, a last one with few tiles `least` at the least (fewer CUs at work run faster).
// Measured for 2048 k (us): 64 tiles of 256 x 256 42, 256 as 49; of 192 x 256 64 tiles 34.5, 224 40.7; of
// 128 x 128 128 tiles 20.9, 256 27, 512 35; of 64 x 64 256 tiles 16.6, 512 22, 1024 28.9, 2048 54.
inline double gemm_rounds(int64_t tiles, int slots, double full, double least) {
  const int64_t whole = tiles / slots, rest = tiles % slots;
  return whole * full + (rest ? least + (full - least) * rest / slots : 0.0);
}
// The tile for that: 256, 192 (by 256 columns), 128 or 64, or for small products, whose time is their steps'
// latency, 64 x 64 with the k shared by four groups of waves (16) or 32 x 32 with eight (8), where a CU each has
// a tile: for 2048 k 72 tiles of 16 12.0 us, the same in 240 tiles of 8 9.3. tiles(of, BM, BN): how many there are.
inline int gemm_class(int64_t (*tiles)(const void *, int, int), const void *of, int64_t steps) {
  if (tiles(of, 32, 32) <= 256 && steps >= 16) return 8;
  if (tiles(of, 64, 64) <= 256 && steps >= 8) return 16;
  const double l = gemm_rounds(tiles(of, 256, 256), 256, 1.0, 0.85), k = gemm_rounds(tiles(of, 192, 256), 256, 0.78, 0.66),
               m = gemm_rounds(tiles(of, 128, 128), 512, 0.68, 0.42), q = gemm_rounds(tiles(of, 64, 64), 1024, 0.52, 0.35);
  if (k < l && k < m && k < q) return 192;
  return l <= m && l <= q ? 256 : m <= q ? 128 : 64;
}
template <class T>
struct TileTag {
  using type = T;
};
// Workgroups for that many tiles where `most` run at a time.
inline int gemm_grid(int64_t tiles, int most) { return (int)((tiles < most ? tiles : most) + 7) / 8 * 8; }

}  // namespace nf4moe
