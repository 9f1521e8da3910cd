// The losses of a vocabulary head, softmax cross entropy and distillation from a teacher's top
// logits, without ever storing the logits l = x W^T [T, V].
//
// Forward: a tile of logits is reduced in registers to a maximum and a sum of exponentials a row
// (k_head_stats, k_head_few), these pairs are joined row by row (k_head_join):
//   lse = log sum_v exp(l_v / tau);  CE: loss = lse - l_label
//   distillation: q = softmax of the teacher's given logits / tau (k_head_entries),
//   loss = tau^2 sum_j q_j (log q_j - l_{id_j} / tau + lse)
// The logits that the loss names are picked out of the tile that holds them.
// Backward, by pieces of the vocabulary that the last-level cache can hold: the tile's logits again,
//   P = dloss (exp(l - lse) - [v is the label])         or dloss tau (softmax - q)
// rounded to bf16 (half a step of 2^-8 of each value, no more than the gradients' own
// rounding; P is the operand of two bf16 products; up to kTwoParts rows it has two parts, which
// leave 2^-17), then dx += P W and dW = P^T x. Of more rows P holds dloss / unit, and the products' sums are
// multiplied by unit in fp32: in a mean loss, where dloss is the same in every row, a label's entry is then all
// but a power of two and not dloss, whose rounding would be every row's (1020 rows of 1 / 1020: both
// gradients off by 1.06 2^-8 in the 2-norm with it, by 0.6 2^-8 at most so).
// All of it is bound by the matrix cores and their power; a handful of rows by the reading of W.
//
// Measured, us, with H 2048, V 50304: 4096 rows forward 643 to 663 (1270 to 1310 TFLOP/s), both gradients
// 2010 to 2120 (1195 to 1260 of 2532 GFLOP). The head's 17 rows with V 32003 (131 MB): 28 + 4 to join. Distillation,
// k 64, 2048 rows, H 2880: 505 to 522, of which the teacher's entries 12 and the joining 6; its gradient dx of 515
// rows, H 1024, V 32003: 111 to 114 for 5 (entries) + 58 (P) + 39 (product) + 9 (its 21 slices).
//
// Exponentials are taken in powers of two: z = l log2(e) / tau. A row's maximum m is rounded, its terms
// 2^(z - m) and what a loss needs of it, m - z, come from one fma of l each: lse - l / tau = (m - z + log2 s) ln 2, where
// a row sure of its label loses nothing (apart, lse rounded at a logit of 40, they left 4 10^-6, on either side of 0).
#include "dense.h"
#include "gemm16.h"
#include "internal.h"

namespace nf4moe {

namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kLowest = -3.402823466e38f;

// Adds (m2, s2) to (m, s): sums of 2^(z - m). m may be -inf with s = 0. m may be a product, whose fma with -top would
// not be 0 where it is the top: its rounding would be in s twice.
__device__ inline void join_stats(float &m, float &s, float m2, float s2) {
#pragma clang fp contract(off)
  const float top = fmaxf(fmaxf(m, m2), kLowest);
  s = __builtin_fmaf(s, __builtin_amdgcn_exp2f(m - top), s2 * __builtin_amdgcn_exp2f(m2 - top));
  m = top;
}

template <class T>
struct HeadPlace : GemmTiles {
  const HeadArgs &p;
  __device__ HeadPlace(const HeadArgs &a, int b, int nb)
      : GemmTiles{b, nb, (int)((a.T + T::BM - 1) / T::BM), (int)((a.vn + T::BN - 1) / T::BN), 1, a.H}, p(a) {}
  // the tile's first row, and its first column of the piece
  __device__ bool at(int r, int64_t &m0, int64_t &n0) const {
    int m, n, slice;
    if (!find(r, m, n, slice)) return false;
    m0 = (int64_t)m * T::BM, n0 = (int64_t)n * T::BN;
    return true;
  }
  __device__ bool operator()(int r, typename T::X &x, typename T::Y &y, GemmRange &k) const {
    int64_t m0, n0;
    if (!at(r, m0, n0)) return false;
    x.init(p.x, p.H, m0, p.T);
    y.init(p.w + p.v0 * p.H, p.H, n0, p.vn);
    k = {0, p.H};
    return true;
  }
};

// The teacher's entries of 16 MB rows in the COLS columns from v on (COLS divides kHeadChunk, v is a
// multiple of it): the lists of MB blocks of 16 rows, their first 64 entries in a register each, asked for
// together, since every one of these loads has the whole latency of memory.
template <int MB, int COLS>
struct TileEntries {
  uint32_t w[MB];
  int first[MB], n[MB];
  int at;   // of v in its chunk
  __device__ void load(const HeadArgs &p, int lane, int64_t row0, int64_t v) {
    const int64_t chunks = (p.V + kHeadChunk - 1) / kHeadChunk;
    at = (int)(v % kHeadChunk);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int64_t block = (row0 >> 4) + mb;
      first[mb] = n[mb] = 0;
      if (16 * block < p.T) {
        const int32_t *off = p.offsets + block * (chunks + 1) + v / kHeadChunk;
        first[mb] = off[0], n[mb] = off[1] - off[0];
      }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      w[mb] = 0;
      if (lane < n[mb]) w[mb] = p.list[((row0 >> 4) + mb) * 16 * p.k + first[mb] + lane];
    }
  }
  // f(row of the block, column of COLS, entry j) where word `of` is one of these columns
  template <class F>
  __device__ void one(uint32_t of, F &&f) const {
    const int col = (int)(of & 127) - at;
    if (col >= 0 && col < COLS) f((int)(of >> 7 & 15), col, (int)(of >> 11));
  }
  // those of block mb past the first 64
  template <class F>
  __device__ void rest(const HeadArgs &p, int lane, int64_t row0, int mb, F &&f) const {
    for (int e = 64 + lane; e < n[mb]; e += 64) one(p.list[((row0 >> 4) + mb) * 16 * p.k + first[mb] + e], f);
  }
  template <class F>
  __device__ void each(const HeadArgs &p, int lane, int64_t row0, int mb, F &&f) const {
    if (lane < n[mb]) one(w[mb], f);
    rest(p, lane, row0, mb, f);
  }
};

template <class T, bool TEACH>
__global__ __launch_bounds__(T::THREADS, T::WAVES_SIMD) void k_head_stats(HeadArgs p) {
  constexpr int COLS = 16 * T::NB;   // a wave's
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const HeadPlace<T> place(p, blockIdx.x, gridDim.x);
  int64_t m0, n0;
  if (!place.at(0, m0, n0)) return;
  T t;
  t.run(lds, nullptr, place, [&](int r) __attribute__((always_inline)) {
    place.at(r, m0, n0);
    n0 += T::cols_at();
    const int lane = epilogue_lane(), left = (int)(p.V - n0 < COLS ? p.V - n0 : COLS);   // columns that exist
    if (left <= 0) return;   // the wave
    const float c = kLog2e / p.tau;
    [[maybe_unused]] TileEntries<T::MB, COLS> entries;
    [[maybe_unused]] int32_t id[T::MB];
    if constexpr (TEACH) {
      entries.load(p, lane, m0 + T::row_at(0), n0);
    } else {   // asked for together
#pragma unroll
      for (int mb = 0; mb < T::MB; ++mb) {
        const int64_t row = m0 + T::row_at(mb) + (lane & 15);
        id[mb] = p.ids[row < p.T ? row : p.T - 1];
      }
    }
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int64_t row0 = m0 + T::row_at(mb), row = row0 + (lane & 15);
      if (row0 >= p.T) break;   // the wave
      if constexpr (!TEACH) {   // the labels' logits, each by the one lane that has it
        const int64_t at = (int64_t)id[mb] - n0;
        const int want = row < p.T && at >= 0 && at < left ? (int)at : -1;
        if (__any(want >= 0)) {
#pragma unroll
          for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (want == T::col_of(lane, nb) + i) p.picked[row] = t.acc[nb][mb][i];
        }
      } else {   // half of the columns at a time as fp32 rows in the wave's own LDS, in 16-byte pieces
        using Row = BlockRow<COLS>;
        char *mine = T::scratch(lds);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int nb = 0; nb < T::NB / 2; ++nb)
            *reinterpret_cast<f32x4_t *>(mine + Row::place(lane & 15, 4 * nb + (lane >> 4))) = t.acc[half * T::NB / 2 + nb][mb];
          wave_lds_order();
          entries.each(p, lane, m0 + T::row_at(0), mb, [&](int er, int col, int j) {
            const int at = col - half * COLS / 2;
            if (at >= 0 && at < COLS / 2)
              p.logits[(row0 + er) * p.k + j] = *reinterpret_cast<const float *>(mine + Row::place(er, at >> 2) + 4 * (at & 3));
          });
          wave_lds_order();
        }
      }
      if (left < COLS) {
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (T::col_of(lane, nb) + i >= left) t.acc[nb][mb][i] = -__builtin_inff();
      }
      float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, t.acc[nb][mb][i]);
      m *= c;
      const float top = fmaxf(m, kLowest);
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s += __builtin_amdgcn_exp2f(__builtin_fmaf(t.acc[nb][mb][i], c, -top));
      join_stats(m, s, __shfl_xor(m, 16, kWave), __shfl_xor(s, 16, kWave));
      join_stats(m, s, __shfl_xor(m, 32, kWave), __shfl_xor(s, 32, kWave));
      if (lane < 16 && row < p.T) p.stats[n0 / COLS * p.T + row] = make_float2(m, s);
    }
  });
}

// Up to 16 MB rows: a workgroup takes 64 columns, a chunk of statistics, a wave 16 of them.
template <int MB, bool TEACH>
__global__ __launch_bounds__(256) void k_head_few(HeadArgs p) {
  using F = FewStream<6, 0>;   // (144 KB for two workgroups a CU)
  __shared__ __attribute__((aligned(16))) char lds[F::LDS];
  const int64_t n0 = (int64_t)blockIdx.x * 64;
  const int T = (int)p.T;
  typename F::X x;
  typename F::Y y;
  x.init(p.x, p.H, 0, p.T);
  y.init(p.w, p.H, n0, p.V);
  f32x4_t acc[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) acc[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int wave = F::X::wave(), lane = threadIdx.x & 63;
  F::run(lds, p.H, x, y, [&](const char *xs, const char *ys) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const bf16x8_t fy = F::Y::frag(ys, wave, kk);
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fy, F::X::frag(xs, m, kk), acc[m], 0, 0, 0);
    }
  });
  const int64_t c0 = n0 + 16 * wave;
  const int left = (int)(p.V - c0 < 16 ? p.V - c0 : 16), col = 4 * (lane >> 4);
  const float scale = kLog2e / p.tau;
  float2 *stats = reinterpret_cast<float2 *>(lds + 4 * 1024);   // [4][16 MB], behind a kilobyte a wave
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t row0 = 16 * mb, row = row0 + (lane & 15);
    f32x4_t v = acc[mb];
    if constexpr (!TEACH) {
      if (row < T) {
        const int64_t want = (int64_t)p.ids[row] - c0 - col;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (want == j && col + j < left) p.picked[row] = v[j];
      }
    } else if (row0 < T && left > 0) {
      f32x4_t *mine = reinterpret_cast<f32x4_t *>(lds) + wave * 64;
      mine[lane] = v;
      wave_lds_order();
      TileEntries<1, 16> entries;
      entries.load(p, lane, row0, c0);
      entries.each(p, lane, row0, 0, [&](int er, int c, int j) {
        p.logits[(row0 + er) * p.k + j] = reinterpret_cast<const float *>(mine + (c >> 2) * 16 + er)[c & 3];
      });
      wave_lds_order();
    }
    float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (col + j >= left) v[j] = -__builtin_inff();
      m = fmaxf(m, v[j]);
    }
    m *= scale;
    const float top = fmaxf(m, kLowest);
#pragma unroll
    for (int j = 0; j < 4; ++j) s += __builtin_amdgcn_exp2f(__builtin_fmaf(v[j], scale, -top));
    join_stats(m, s, __shfl_xor(m, 16, kWave), __shfl_xor(s, 16, kWave));
    join_stats(m, s, __shfl_xor(m, 32, kWave), __shfl_xor(s, 32, kWave));
    if (lane < 16) stats[wave * 16 * MB + row] = make_float2(m, s);
  }
  lds_barrier();
  const int r = threadIdx.x;
  if (r >= 16 * MB || r >= T) return;
  float2 a = stats[r];
#pragma unroll
  for (int n = 1; n < 4; ++n) join_stats(a.x, a.y, stats[n * 16 * MB + r].x, stats[n * 16 * MB + r].y);
  p.stats[(int64_t)blockIdx.x * p.T + r] = a;
}

// R rows a workgroup of W waves, 64 W / R threads each: the chunks' pairs to lse, and the loss.
template <int R, int W>
__global__ __launch_bounds__(64 * W) void k_head_join(HeadArgs p, int chunks) {
  constexpr int PARTS = 64 * W / R;   // threads of a row
  static_assert(R <= 64, "rows of a wave");
  __shared__ float2 red[2][W][R];
  const int r = threadIdx.x % R, part = threadIdx.x / R, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * R + r;
  const bool live = row < p.T;
  float m = -__builtin_inff(), s = 0.0f;
  if (live) {
#pragma unroll 8
    for (int n = part; n < chunks; n += PARTS) {
      const float2 v = p.stats[(int64_t)n * p.T + row];
      join_stats(m, s, v.x, v.y);
    }
  }
#pragma unroll
  for (int d = R; d < 64; d *= 2) join_stats(m, s, __shfl_xor(m, d, kWave), __shfl_xor(s, d, kWave));
  if (lane < R) red[0][wave][r] = make_float2(m, s);
  lds_barrier();
  m = red[0][0][r].x, s = red[0][0][r].y;
#pragma unroll
  for (int w = 1; w < W; ++w) join_stats(m, s, red[0][w][r].x, red[0][w][r].y);
  const float log_s = log2f(s), lse = (m + log_s) * kLn2, c = kLog2e / p.tau;
  const auto above = [&](float l) { return (__builtin_fmaf(-l, c, m) + log_s) * kLn2; };   // lse - l / tau
  if (p.k == 0) {
    if (part == 0 && live) {
      const int32_t id = p.ids[row];
      p.loss[row] = id >= 0 && id < p.V ? above(p.picked[row]) : 0.0f;
      p.lse[row] = lse;
    }
    return;
  }
  float sum = 0.0f, any = 0.0f;
  if (live) {
    for (int j = part; j < p.k; j += PARTS) {
      const float q = p.q[row * p.k + j];
      if (q == 0.0f) continue;
      any = 1.0f;
      sum += q * (logf(q) + above(p.logits[row * p.k + j]));
    }
  }
#pragma unroll
  for (int d = R; d < 64; d *= 2) sum += __shfl_xor(sum, d, kWave), any += __shfl_xor(any, d, kWave);
  if (lane < R) red[1][wave][r] = make_float2(sum, any);
  lds_barrier();
  if (part == 0 && live) {
    for (int w = 1; w < W; ++w) sum += red[1][w][r].x, any += red[1][w][r].y;
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

// Places of a row's table of ids: a power of two, half of them free.
__host__ __device__ inline int table_size(int k) {
  int n = 64;
  while (n < 2 * k) n *= 2;
  return n;
}
// q [k] of a row from the teacher's logits, by a wave with `val` and `ids` [k] and `table` [table_size(k)]
// of its own in LDS. Entries outside the vocabulary count for nothing, an id's later occurrences add to
// its first; a row without an entry above -inf has all zeros. Also zeros the logits of entries outside
// and leaves their ids as -1. An id that occurs twice is noticed by a table of ids with open places (which of
// its entries is the place's is open, whether there are two is not), and only for it the wave goes through all.
__device__ inline void teacher_row(const HeadArgs &p, int64_t row, int lane, float *val, int32_t *ids, uint32_t *table) {
  constexpr uint32_t kTwice = 0x80000000u;
  const int64_t base = row * p.k;
  const int places = table_size(p.k), shift = __clz(places) + 1;   // of a 32-bit hash
  float m = -__builtin_inff();
  bool nan = false;
  for (int j = lane; j < p.k; j += 64) {
    int32_t id = p.ids[base + j];
    float t = p.teacher_bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p.teacher)[base + j])
                             : reinterpret_cast<const float *>(p.teacher)[base + j];
    if (id < 0 || id >= p.V) {
      id = -1, t = -__builtin_inff();
      p.logits[base + j] = 0.0f;
    }
    ids[j] = id, val[j] = t;
    nan |= t != t;
    m = fmaxf(m, t);
  }
  for (int i = lane; i < places; i += 64) table[i] = 0;
  m = wave_max(m);
  nan = __any(nan);
  float sum = 0.0f;
  for (int j = lane; j < p.k; j += 64) {
    const float e = m == -__builtin_inff() ? 0.0f : expf((val[j] - m) / p.tau);
    val[j] = e;
    sum += e;
  }
  sum = wave_sum(sum);
  wave_lds_order();
  auto hash = [&](int32_t id) { return (int)((uint32_t)id * 2654435769u >> shift); };
  for (int j = lane; j < p.k; j += 64) {
    const int32_t id = ids[j];
    if (id < 0) continue;
    for (int at = hash(id);; at = (at + 1) & (places - 1)) {
      const uint32_t was = atomicCAS(&table[at], 0u, (uint32_t)j + 1);
      if (was == 0) break;
      if (ids[(was & ~kTwice) - 1] == id) {
        atomicOr(&table[at], kTwice);
        break;
      }
    }
  }
  wave_lds_order();
  for (int j0 = 0; j0 < p.k; j0 += 64) {
    const int j = j0 + lane;
    const int32_t id = j < p.k ? ids[j] : -1;
    bool twice = false, mine = false;   // its place is shared; it is this entry's
    if (id >= 0) {
      int at = hash(id);
      while (ids[(table[at] & ~kTwice) - 1] != id) at = (at + 1) & (places - 1);   // it is there
      twice = table[at] & kTwice, mine = (table[at] & ~kTwice) == (uint32_t)j + 1;
    }
    const bool none = id < 0 || m == -__builtin_inff();
    if (j < p.k && (nan || !twice || none)) p.q[base + j] = nan && id >= 0 ? __builtin_nanf("") : none ? 0.0f : val[j] / sum;
    for (uint64_t of = __ballot(twice && mine && !nan && !none); of; of &= of - 1) {   // the wave, an id at a time
      const int32_t want = __shfl(id, __builtin_ctzll(of), kWave);
      float e = 0.0f;
      int first = p.k;
      for (int i = lane; i < p.k; i += 64)
        if (ids[i] == want) e += val[i], first = first < i ? first : i;
      e = wave_sum(e);
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_xor(first, d, kWave);
        first = first < other ? first : other;
      }
      for (int i = lane; i < p.k; i += 64)
        if (ids[i] == want) p.q[base + i] = i == first ? e / sum : 0.0f;
    }
  }
  wave_lds_order();
}

// unit: the significand, 1 .. 2, of dloss tau in the first row where it is a normal number (no such row: 1). A power
// of two is the quotient where dloss is the same, and dloss / unit keeps dloss's range. By a workgroup of
// 1024 threads, 8192 rows a round, the first of them in nearly every call: 2.4 us by itself for 131 rows, 5 for 4096, none
// beside the entries.
__device__ inline void head_unit(const HeadArgs &p) {
  constexpr int U = 8;
  __shared__ int least[2][16];
  const int t = threadIdx.x, T = (int)p.T;   // (2^25 at the most)
  int turn = 0;
  for (int r0 = 0; r0 < T; r0 += U * 1024, turn ^= 1) {
    int first = T;
#pragma unroll
    for (int i = U - 1; i >= 0; --i) {
      const int row = r0 + i * 1024 + t, in = row < T ? row : T - 1;
      const uint32_t size = __float_as_uint(p.dloss[in] * p.tau) & 0x7fffffffu;
      if (row < T && row_on(p, in) && size >= 0x00800000u && size < 0x7f800000u) first = row;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) first = min(first, __shfl_xor(first, d, kWave));
    if ((t & 63) == 0) least[turn][t >> 6] = first;
    lds_barrier();   // (a place is written again two rounds on, behind the next round's barrier)
#pragma unroll
    for (int w = 0; w < 16; ++w) first = min(first, least[turn][w]);
    if (first < T) {   // the whole workgroup
      if (t == 0) *p.unit = __uint_as_float((__float_as_uint(p.dloss[first] * p.tau) & 0x007fffffu) | 0x3f800000u);
      return;
    }
  }
  if (t == 0) *p.unit = 1.0f;
}

__global__ __launch_bounds__(1024) void k_head_unit(HeadArgs p) { head_unit(p); }

// A workgroup 16 rows, a wave one of them: the teacher's probabilities (forward), and the rows' entries by
// chunk of kHeadChunk columns (counts, a scan, places). BACK: those with a probability; else those with an
// id in the vocabulary. Within a chunk their order is open: each writes to a place of its own.
// 2048 rows of 64 entries 12 us (every id against every other: 15), 17 of 512 37 (405), of 1024 140 (2100).
constexpr int kEntryThreads = 1024;
// LDS words of a row: ids, and for the forward values and the table.
__host__ __device__ inline int entry_words(int k, bool back) { return back ? k : 2 * k + table_size(k); }
// Rows that are in LDS at a time, beside the counts of 2^21 / kHeadChunk chunks at the most.
inline int entry_rows(int k, int64_t chunks, bool back) {
  int rows = 16;
  while (4 * (chunks + (int64_t)rows * entry_words(k, back)) > (159 << 10)) rows /= 2;
  return rows;
}
template <bool BACK>
__global__ __launch_bounds__(kEntryThreads) void k_head_entries(HeadArgs p, int rows) {
  if constexpr (BACK) {
    static_assert(kEntryThreads == 1024, "the last workgroup, one more than the rows need where P leaves out a unit");
    if ((int64_t)blockIdx.x * 16 >= p.T) return head_unit(p);
  }
  extern __shared__ int32_t shared[];   // [chunks], [rows][entry_words]
  __shared__ int32_t total[kEntryThreads / 64];
  const int t = threadIdx.x, w = t >> 6, lane = t & 63;
  const int chunks = (int)((p.V + kHeadChunk - 1) / kHeadChunk), each = (chunks + kEntryThreads - 1) / kEntryThreads;
  int32_t *count = shared, *ids = shared + chunks + w * entry_words(p.k, BACK);
  const int64_t row0 = (int64_t)blockIdx.x * 16, row = row0 + w, base = row * p.k;
  if constexpr (!BACK) {
    if (w < rows)
      for (int64_t r = row; r < row0 + 16 && r < p.T; r += rows)
        teacher_row(p, r, lane, reinterpret_cast<float *>(ids + p.k), ids, reinterpret_cast<uint32_t *>(ids + 2 * p.k));
  }
  for (int i = t; i < chunks; i += kEntryThreads) count[i] = 0;
  lds_barrier();
  const int n = row < p.T ? p.k : 0;
  const bool held = !BACK && rows == 16;   // the wave's row is in its LDS
  auto id_of = [&](int j) {
    if (held) return (int)ids[j];
    const int32_t id = p.ids[base + j];
    return id < 0 || id >= p.V || (BACK && p.q[base + j] == 0.0f) ? -1 : (int)id;
  };
  for (int j = lane; j < n; j += 64) {
    const int id = id_of(j);
    if (BACK) ids[j] = id;
    if (id >= 0) atomicAdd(&count[id / kHeadChunk], 1);
  }
  lds_barrier();
  int sum = 0;
  for (int i = t * each; i < (t + 1) * each && i < chunks; ++i) sum += count[i];
  int upto = sum;   // in the wave, then over the waves
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d, kWave);
    upto += lane >= d ? v : 0;
  }
  if (lane == 63) total[w] = upto;
  lds_barrier();
  for (int i = 0; i < w; ++i) upto += total[i];
  int at = upto - sum;
  int32_t *off = p.offsets + (int64_t)blockIdx.x * (chunks + 1);
  for (int i = t * each; i < (t + 1) * each && i < chunks; ++i) {
    const int v = count[i];
    off[i] = at, count[i] = at;
    at += v;
  }
  if (t == kEntryThreads - 1) off[chunks] = upto;
  lds_barrier();
  uint32_t *list = p.list + row0 * p.k;
  for (int j = lane; j < n; j += 64) {
    const int id = BACK ? (int)ids[j] : id_of(j);
    if (id >= 0) list[atomicAdd(&count[id / kHeadChunk], 1)] = (uint32_t)j << 11 | (uint32_t)w << 7 | (uint32_t)(id % kHeadChunk);
  }
}

// FEW: up to kTwoParts rows, P in two parts and x twice.
template <class T, bool TEACH, bool FEW>
__global__ __launch_bounds__(T::THREADS, T::WAVES_SIMD) void k_head_piece(HeadArgs p) {
  constexpr int COLS = 16 * T::NB;   // a wave's
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  if constexpr (FEW) {
    const int row16 = p.H / 8, n = (int)p.T * row16;   // 16-byte pieces
    for (int i = (int)blockIdx.x * T::THREADS + threadIdx.x; p.x2 && p.v0 == 0 && i < n; i += (int)gridDim.x * T::THREADS) {
      uint4 v = reinterpret_cast<const uint4 *>(p.x)[i];
      if (!row_on(p, i / row16)) v = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4 *>(p.x2)[i] = v;
      reinterpret_cast<uint4 *>(p.x2)[n + i] = v;
    }
  }
  const HeadPlace<T> place(p, blockIdx.x, gridDim.x);
  int64_t m0, n0;
  if (!place.at(0, m0, n0)) return;
  T t;
  t.run(lds, nullptr, place, [&](int r) __attribute__((always_inline)) {
    place.at(r, m0, n0);
    n0 += T::cols_at();
    const int lane = epilogue_lane(), left = (int)(p.vn - n0 < COLS ? p.vn - n0 : COLS);
    if (left <= 0) return;   // the wave
    const float c = kLog2e / p.tau, unit = FEW ? 1.0f : *p.unit;
    const BlockRow<COLS> out{T::scratch(lds), lane};
    // an entry's P, from its logit in fp32
    [[maybe_unused]] auto entry_value = [&](int64_t row, int j) __attribute__((always_inline)) {
      const int64_t e = row * p.k + j;
      if (!row_on(p, row)) return 0.0f;
      return p.dloss[row] * p.tau / unit * (__builtin_amdgcn_exp2f(p.logits[e] * c - p.lse[row] * kLog2e) - p.q[e]);
    };
    [[maybe_unused]] TileEntries<T::MB, COLS> entries;
    [[maybe_unused]] float value[T::MB];
    [[maybe_unused]] int32_t id[T::MB];
    float dloss[T::MB], row_lse[T::MB];   // asked for together
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int64_t row = m0 + T::row_at(mb) + (lane & 15), in = row < p.T ? row : p.T - 1;
      if constexpr (!TEACH) id[mb] = p.ids[in];
      dloss[mb] = p.dloss[in], row_lse[mb] = p.lse[in];
    }
    if constexpr (TEACH) {
      entries.load(p, lane, m0 + T::row_at(0), p.v0 + n0);
#pragma unroll
      for (int mb = 0; mb < T::MB; ++mb) {
        value[mb] = 0.0f;
        if (lane < entries.n[mb])
          value[mb] = entry_value(m0 + T::row_at(mb) + (entries.w[mb] >> 7 & 15), (int)(entries.w[mb] >> 11));
      }
    }
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int64_t row0 = m0 + T::row_at(mb), row = row0 + (lane & 15);
      if (row0 >= p.T) break;   // the wave
      bool on = row < p.T;
      int want = -1;
      if constexpr (TEACH) {
        on = on && row_lse[mb] != __builtin_inff();
      } else {
        on = on && id[mb] >= 0 && id[mb] < p.V;
        const int64_t at = (int64_t)id[mb] - p.v0 - n0;
        want = on && at >= 0 && at < left ? (int)at : -1;
      }
      const float coef = on ? dloss[mb] * p.tau / unit : 0.0f, lse = on ? row_lse[mb] * kLog2e : 0.0f;
      // the rows that count in dw's product, by the wave that has the vocabulary's first columns
      const uint64_t rows_on = __ballot(on);
      if (p.live && p.v0 + n0 == 0 && lane == 0) reinterpret_cast<uint16_t *>(p.live)[row0 >> 4] = (uint16_t)rows_on;
      const bool some = !TEACH && __any(want >= 0), all = __all(on) && left == COLS;
      [[maybe_unused]] uint2 low[T::NB];
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_exp2f(t.acc[nb][mb][j] * c - lse);
        if (some) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] -= want == T::col_of(lane, nb) + j ? 1.0f : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= coef;
        if (!all) {   // rows without a gradient and columns past the vocabulary, whatever they hold
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = on && T::col_of(lane, nb) + j < left ? v[j] : 0.0f;
        }
        if constexpr (FEW) low[nb] = pack4(bf16_rest(v[0]), bf16_rest(v[1]), bf16_rest(v[2]), bf16_rest(v[3]));
        out.put(T::col_of(lane, nb), pack4(v[0], v[1], v[2], v[3]));
      }
      if constexpr (TEACH) {   // the entries' places
        wave_lds_order();
        if (lane < entries.n[mb])
          entries.one(entries.w[mb], [&](int er, int col, int) { *out.one(er, col) = (uint16_t)f32_to_bf16_rne(value[mb]); });
        entries.rest(p, lane, m0 + T::row_at(0), mb, [&](int er, int col, int j) {
          *out.one(er, col) = (uint16_t)f32_to_bf16_rne(entry_value(row0 + er, j));
        });
      }
      uint16_t *to = p.P + row0 * p.vp + n0;
      out.out(to, p.vp, p.T - row0, p.vp - n0);
      if constexpr (FEW) {
        auto rest_of = [](float v) { return (uint16_t)f32_to_bf16_rne(bf16_rest(v)); };
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) out.put(T::col_of(lane, nb), low[nb]);
        if constexpr (TEACH) {
          wave_lds_order();
          if (lane < entries.n[mb])
            entries.one(entries.w[mb], [&](int er, int col, int) { *out.one(er, col) = rest_of(value[mb]); });
          entries.rest(p, lane, m0 + T::row_at(0), mb,
                       [&](int er, int col, int j) { *out.one(er, col) = rest_of(entry_value(row0 + er, j)); });
        }
        out.out(to + p.T * p.vp, p.vp, p.T - row0, p.vp - n0);
      }
    }
  });
}

template <bool BACK>
hipError_t launch_entries(const HeadArgs &a, hipStream_t s) {
  const int64_t chunks = cdiv(a.V, kHeadChunk);
  const int rows = entry_rows(a.k, chunks, BACK);
  hipLaunchKernelGGL(k_head_entries<BACK>, dim3((unsigned)cdiv(a.T, 16) + (BACK && a.unit ? 1 : 0)), dim3(kEntryThreads),
                     4 * (chunks + (int64_t)rows * entry_words(a.k, BACK)), s, a, rows);
  return hipGetLastError();
}

struct HeadSize {
  int64_t T, V;
};
int64_t head_tile_count(const void *size, int bm, int bn) {
  const HeadSize &a = *static_cast<const HeadSize *>(size);
  return cdiv(a.T, bm) * cdiv(a.V, bn);
}
// f(the tile of a call)
template <class F>
void by_head_tile(int64_t T, int64_t V, int H, F &&f) {
  const HeadSize size{T, V};
  int c = gemm_class(head_tile_count, &size, cdiv(H, kGemmBK));
  if (T <= kTwoParts && c > 64) c = 64;
  switch (c) {
    case 256: return f(TileTag<GemmTile<4, 8, 4, 2>>());
    case 192: return f(TileTag<GemmTile<3, 8, 4, 2>>());
    case 128: return f(TileTag<GemmTile<4, 4, 2, 2>>());
    case 64: return f(TileTag<GemmTile<2, 2, 2, 2>>());
    case 16: return f(TileTag<GemmTile<2, 2, 2, 2, false, false, 0, false, 4>>());
    default: return f(TileTag<GemmTile<1, 2, 2, 1, false, false, 0, false, 8>>());
  }
}
template <class T>
dim3 head_grid(int64_t rows, int64_t cols) {
  const int64_t tiles = cdiv(rows, T::BM) * cdiv(cols, T::BN);
  return dim3(T::KS > 1 ? (unsigned)cdiv(tiles, 8) * 8 : gemm_grid(tiles, T::MOST));
}

// The form for few rows, where half of the CUs have columns of it at least: 17 rows, H 4096, stream and tiles in us:
// V 4000 20.6 and 16.5, 8000 20.7 and 20.7, 12000 21.3 and 27.6, 32003 47.5 and 58.9.
bool head_few(int64_t T, int64_t V) { return T <= 32 && V > 64 * 128; }

}  // namespace

int64_t head_stat_chunks(int64_t T, int64_t V, int H) {
  if (head_few(T, V)) return cdiv(V, 64);
  int64_t n = 0;
  by_head_tile(T, V, H, [&](auto tile) { n = cdiv(V, 16 * decltype(tile)::type::NB); });
  return n;
}

hipError_t launch_head_forward(const HeadArgs &args, hipStream_t s) {
  HeadArgs a = args;
  a.v0 = 0, a.vn = a.V;
  if (a.k) {
    const hipError_t e = launch_entries<false>(a, s);
    if (e != hipSuccess) return e;
  }
  if (head_few(a.T, a.V)) {
    const dim3 grid((unsigned)cdiv(a.V, 64)), block(256);
    const auto go = [&](auto mb) {
      constexpr int MB = decltype(mb)::value;
      if (a.k) hipLaunchKernelGGL((k_head_few<MB, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((k_head_few<MB, false>), grid, block, 0, s, a);
    };
    if (a.T <= 16) go(std::integral_constant<int, 1>());
    else go(std::integral_constant<int, 2>());
  } else {
    by_head_tile(a.T, a.V, a.H, [&](auto tile) {
      using T = typename decltype(tile)::type;
      const dim3 grid = head_grid<T>(a.T, a.V);
      if (a.k) hipLaunchKernelGGL((k_head_stats<T, true>), grid, dim3(T::THREADS), 0, s, a);
      else hipLaunchKernelGGL((k_head_stats<T, false>), grid, dim3(T::THREADS), 0, s, a);
    });
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int chunks = (int)head_stat_chunks(a.T, a.V, a.H);
  // enough workgroups whatever T, and 64 or 128 bytes of a chunk's pairs each where there are rows for it (2048 rows,
  // V 50304: eight rows 5.0 us, four 6.6; 4096: 7.7, and 16 rows 4.9)
  if (a.T <= 256) hipLaunchKernelGGL((k_head_join<1, 4>), dim3((unsigned)a.T), dim3(256), 0, s, a, chunks);
  else if (a.T <= 2048) hipLaunchKernelGGL((k_head_join<8, 16>), dim3((unsigned)cdiv(a.T, 8)), dim3(1024), 0, s, a, chunks);
  else hipLaunchKernelGGL((k_head_join<16, 4>), dim3((unsigned)cdiv(a.T, 16)), dim3(256), 0, s, a, chunks);
  return hipGetLastError();
}

hipError_t launch_head_prepare(const HeadArgs &a, hipStream_t s) {
  if (a.k) return launch_entries<true>(a, s);
  if (a.unit) hipLaunchKernelGGL(k_head_unit, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_head_piece(const HeadArgs &a, hipStream_t s) {
  by_head_tile(a.T, a.vn, a.H, [&](auto tile) {
    using T = typename decltype(tile)::type;
    const dim3 grid = head_grid<T>(a.T, a.vn);
    if constexpr (T::BM <= 64) {   // (the tiles of few rows)
      if (a.T <= kTwoParts) {
        if (a.k) hipLaunchKernelGGL((k_head_piece<T, true, true>), grid, dim3(T::THREADS), 0, s, a);
        else hipLaunchKernelGGL((k_head_piece<T, false, true>), grid, dim3(T::THREADS), 0, s, a);
        return;
      }
    }
    if (a.k) hipLaunchKernelGGL((k_head_piece<T, true, false>), grid, dim3(T::THREADS), 0, s, a);
    else hipLaunchKernelGGL((k_head_piece<T, false, false>), grid, dim3(T::THREADS), 0, s, a);
  });
  return hipGetLastError();
}

// Columns of a piece: P [rows, piece] in bf16 takes at most 128 MB of the 256 MB last-level cache, so that
// the two products read it from there; whole rounds of 256 tiles where the rows allow (4096 columns for
// 4096 rows), at least 256.
int64_t head_piece(int64_t rows, int64_t V) {
  int64_t n = ((int64_t)1 << 26) / rows;
  if (n >= V) return (V + 255) / 256 * 256;
  n = n >= 4096 ? n / 4096 * 4096 : n / 256 * 256;
  return n < 256 ? 256 : n;
}

}  // namespace nf4moe
