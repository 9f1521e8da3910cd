// Low-rank adapters of many requests or experts beside a shared projection.
//
//   t[r] = A_l x[m(r)],  out[r] = base[r] + s_l B_l t[r]          (l = ids[r])
//   u[r] = s_l B_l^T dy[r],  dx[r] = dx_base[r] + A_l^T u[r]
//   dA_l = sum_r u[r] x[m(r)]^T,  dB_l = s_l sum_r dy[r] t[r]^T
//
// The rank is small (8..128), so every product is bound by the traffic of the
// wide operands (x, base / out, dy, dx), and the matrix cores have room to spare.
// That room buys exactness: t and u stay fp32, and enter the second product as
// the exact sum of three bf16 parts (8 + 8 + 8 significant bits by truncation),
// so nothing but the fp32 additions is rounded before the output.
//
// Rows are grouped by adapter once per call (or once per batch, by the caller): a
// stable counting sort, then a table of tiles of up to 64 rows of one adapter.
#include "ckpt8.h"
#include "internal.h"
#include "train.h"

namespace nf4moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ inline f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
  // 16x16x32: a holds row lane & 15, b column lane & 15, both k = 8 (lane >> 4) ..;
  // c holds column lane & 15, rows 4 (lane >> 4) ..
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Eight fp32 values as three bf16 parts whose sum is the value exactly: each part
// takes the next 8 significant bits by truncation (so a finite value never
// becomes infinite). An infinity or NaN is its own first part, the others 0.
__device__ inline void split3(const float (&v)[8], uint4 &hi, uint4 &mid, uint4 &lo) {
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t b = __float_as_uint(v[i]);
    const bool finite = (b & 0x7f800000u) != 0x7f800000u;
    if (!finite && (b & 0x7fffffu)) b |= 0x400000u;  // a NaN whose payload is in the low half stays one
    h[i] = b;
    const float r = finite ? v[i] - __uint_as_float(b & 0xffff0000u) : 0.0f;
    m[i] = __float_as_uint(r);
    l[i] = __float_as_uint(r - __uint_as_float(m[i] & 0xffff0000u));
  }
  auto top = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); };  // high halves of a, b
  hi = make_uint4(top(h[0], h[1]), top(h[2], h[3]), top(h[4], h[5]), top(h[6], h[7]));
  mid = make_uint4(top(m[0], m[1]), top(m[2], m[3]), top(m[4], m[5]), top(m[6], m[7]));
  lo = make_uint4(top(l[0], l[1]), top(l[2], l[3]), top(l[4], l[5]), top(l[6], l[7]));
}

// ------------------------------------------------------------------ grouping
constexpr int kPlanThreads = 1024;

// Rows of one plan workgroup: 1024, or more where (workgroups) x (bins) would
// exceed 64 K counters, which every workgroup reads.
int plan_rows(int R, int L) {
  const int64_t blocks = cdiv(R, kPlanThreads);
  const int64_t per = cdiv(blocks * (L + 1), 65536);
  return (int)(kPlanThreads * (per < 1 ? 1 : per));
}

__device__ inline int bin_of(int id, int L) { return id < 0 || id >= L ? L : id; }

constexpr int kPrepareThreads = 256;
// The row counters of every bin per plan workgroup.
__global__ __launch_bounds__(kPrepareThreads) void k_plan_hist(const int32_t *__restrict__ ids, int R, int L, int per,
                                                               int32_t *__restrict__ hist) {
  extern __shared__ int32_t cnt[];
  for (int b = threadIdx.x; b <= L; b += kPrepareThreads) cnt[b] = 0;
  __syncthreads();
  const int r0 = blockIdx.x * per, r1 = min(R, r0 + per);
  for (int r = r0 + (int)threadIdx.x; r < r1; r += kPrepareThreads) atomicAdd(&cnt[bin_of(ids[r], L)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b <= L; b += kPrepareThreads) hist[(int64_t)blockIdx.x * (L + 1) + b] = cnt[b];
}

// Turned copies of the adapters' weights for the backward: [L][P][Q] -> [L][Q][P]. A
// thread turns 8 x 8 values in registers: 16-byte loads along Q, 16-byte stores
// along P, the rank's dimension fastest over the lanes.
struct TurnArgs {
  const uint16_t *in;
  uint16_t *out;
  int P, Q;
  bool p_is_rank;
};
// Rows (2 i, 2 i + 1) of column k of an 8 x 8 block of 16-bit values as one word.
__device__ inline void turn_8x8(const uint4 (&row)[8], uint32_t (&blk)[4][8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u[4] = {row[2 * i].x, row[2 * i].y, row[2 * i].z, row[2 * i].w};
    const uint32_t w[4] = {row[2 * i + 1].x, row[2 * i + 1].y, row[2 * i + 1].z, row[2 * i + 1].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      blk[i][2 * k] = __builtin_amdgcn_perm(w[k], u[k], 0x05040100u);
      blk[i][2 * k + 1] = __builtin_amdgcn_perm(w[k], u[k], 0x07060302u);
    }
  }
}
template <int THREADS>
__device__ inline void turn_block(const TurnArgs &a, int l, int block) {
  const int p8 = a.P / 8, q8 = a.Q / 8;
  const int i = block * THREADS + (int)threadIdx.x;
  if (i >= p8 * q8) return;
  const int p = 8 * (a.p_is_rank ? i % p8 : i / q8), q = 8 * (a.p_is_rank ? i / p8 : i % q8);
  const int64_t base = (int64_t)l * a.P * a.Q;
  uint4 row[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) row[k] = load16(a.in + base + (int64_t)(p + k) * a.Q + q);
  uint32_t blk[4][8];
  turn_8x8(row, blk);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    store16(a.out + base + (int64_t)(q + k) * a.P + p, make_uint4(blk[0][k], blk[1][k], blk[2][k], blk[3][k]));
}

// Block i of the turned copies: per adapter b0 blocks of the first array, then b1 of the
// second (0 where there is none).
struct TurnPair {
  TurnArgs t0, t1;
  int b0, b1;
};
template <int THREADS>
__device__ inline void turn_blocks(const TurnPair &t, int i) {
  const int l = i / (t.b0 + t.b1), block = i % (t.b0 + t.b1);
  if (block < t.b0) turn_block<THREADS>(t.t0, l, block);
  else turn_block<THREADS>(t.t1, l, block - t.b0);
}

__global__ __launch_bounds__(kPrepareThreads) void k_turn(TurnPair turn) { turn_blocks<kPrepareThreads>(turn, (int)blockIdx.x); }

// Exclusive prefixes of four counts over the workgroup's threads in order; totals in *sum.
__device__ inline int4 block_prefix4(int4 v, int4 *wsum, int4 *sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int4 x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int4 y = make_int4(__shfl_up(x.x, d, kWave), __shfl_up(x.y, d, kWave), __shfl_up(x.z, d, kWave), __shfl_up(x.w, d, kWave));
    if (lane >= d) x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
  }
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  int4 before = make_int4(0, 0, 0, 0), all = make_int4(0, 0, 0, 0);
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const int4 s = wsum[w];
    if (w < wave) before.x += s.x, before.y += s.y, before.z += s.z, before.w += s.w;
    all.x += s.x, all.y += s.y, all.z += s.z, all.w += s.w;
  }
  *sum = all;
  return make_int4(before.x + x.x - v.x, before.y + x.y - v.y, before.z + x.z - v.z, before.w + x.w - v.w);
}

// One workgroup per `per` rows. Each finds, for every bin, where its own rows of
// that bin begin (all counters of the earlier workgroups and bins), then places
// its rows in order, 1024 at a time: ranks inside a wave by ballots, then the
// waves' counts of each bin in wave order, so the order is stable. Workgroup 0 also
// writes the chunk table; all share the tile table. Bound by the latency of a chain of
// barriers, 6 to 10 us up to 32768 rows of 64 adapters, not by bytes.
//
// The counters come from k_plan_hist, or for few rows every workgroup counts all of them
// itself. Workgroups behind these turn the backward's weights, those of all L adapters,
// beside the grouping; the next launch waits for both. us, two launches against one: 4099 rows of 6 adapters 2.4 + 5.9 / 7.8, 8192 of 64 2.4 + 10.2 / 12.7,
// 16384 of 64 2.1 + 10.3 / 15.9.
constexpr int kSelfCount = 8192;
constexpr int kWaveBins = 1024;  // up to so many bins the waves' counts have a place each in LDS
__global__ __launch_bounds__(kPlanThreads) void k_plan_scatter(const int32_t *__restrict__ ids, int R, int L, int per,
                                                               int groups, bool self_count, int chunk_rows, AdapterPlan p,
                                                               TurnPair turn) {
  constexpr int W = kPlanThreads / 64;
  __shared__ int32_t next[kMaxAdapters + 1], tot[kMaxAdapters + 1];
  __shared__ union {
    uint16_t count[W][kWaveBins];
    int32_t bins[2][kMaxAdapters + 1];
  } u;
  __shared__ int4 wsum[W];
  auto &wcnt = u.count;
  int32_t *bin_tile = u.bins[0], *bin_row = u.bins[1];  // each bin's first tile and first place
  if ((int)blockIdx.x >= groups) {
    turn_blocks<kPlanThreads>(turn, (int)blockIdx.x - groups);
    return;
  }
  const int tid = threadIdx.x, nb = L + 1;
  const int r0 = blockIdx.x * per, r1 = min(R, r0 + per);
  int b = r0 + tid < r1 ? bin_of(ids[r0 + tid], L) : -1;
  for (int i = tid; i < nb; i += kPlanThreads) next[i] = tot[i] = 0;
  __syncthreads();
  if (self_count) {
    // a wave's rows of its first lane's bin as one addition: neighbours often share one
    auto count = [&](int bin, int32_t *cnt) {
      const int lead = __builtin_amdgcn_readfirstlane(bin);
      const uint64_t same = __ballot(bin == lead);
      if (bin != lead) {
        if (bin >= 0) atomicAdd(&cnt[bin], 1);
      } else if (lead >= 0 && (threadIdx.x & 63) == (unsigned)__builtin_ctzll(same)) {
        atomicAdd(&cnt[lead], __popcll(same));
      }
    };
    for (int base = 0; base < R; base += 4 * kPlanThreads) {
      int bin[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = base + k * kPlanThreads + tid;
        bin[k] = r < R ? bin_of(ids[r], L) : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = base + k * kPlanThreads;  // `per` is a multiple of kPlanThreads: all of these rows are before r0, or none
        if (at < R) count(bin[k], tot);
        if (at < r0) count(bin[k], next);
      }
    }
  } else {
    for (int i = tid; i < nb * groups; i += kPlanThreads) {
      const int32_t c = p.hist[i];
      if (c == 0) continue;
      const int g = i / nb, bin = i % nb;
      atomicAdd(&tot[bin], c);
      if (g < (int)blockIdx.x) atomicAdd(&next[bin], c);
    }
  }
  __syncthreads();
  const int seg = (nb + kPlanThreads - 1) / kPlanThreads, b0 = tid * seg, b1 = min(nb, b0 + seg);  // this thread's bins
  int4 sums = make_int4(0, 0, 0, 0), all;  // rows, tiles, chunks, slots
  for (int i = b0; i < b1; ++i) {
    const int32_t n = tot[i];
    const int32_t c = i < L ? max(1, (n + chunk_rows - 1) / chunk_rows) : 0;
    sums.x += n;
    sums.y += (n + kAdTile - 1) / kAdTile;
    sums.z += c;
    sums.w += c > 1 ? c : 0;
  }
  int4 at = block_prefix4(sums, wsum, &all);
  if (blockIdx.x == 0 && tid == 0) {
    p.counts[0] = all.y;
    p.counts[1] = all.z;
  }
  for (int i = b0; i < b1; ++i) {
    const int32_t n = tot[i];
    next[i] += at.x;
    bin_tile[i] = at.y;
    bin_row[i] = at.x;
    at.y += (n + kAdTile - 1) / kAdTile;
    if (blockIdx.x == 0) {
      if (i < L) {
        const int32_t c = max(1, (n + chunk_rows - 1) / chunk_rows);  // one of no rows where there are none
        p.chunks_of[i] = make_int2(c, at.w);
        for (int32_t k = 0; k < c; ++k)
          p.chunks[at.z++] = make_int4(i, at.x + k * chunk_rows, min(chunk_rows, n - k * chunk_rows), c > 1 ? at.w + k : -1);
        if (c > 1) at.w += c;
      }
    }
    at.x += n;
  }
  __syncthreads();
  // the tile table, every workgroup its share: a tile's bin is the last that begins
  // at or before it (a bin of no rows begins where the next one does)
  for (int i = (int)blockIdx.x * kPlanThreads + tid; i < all.y; i += groups * kPlanThreads) {
    int lo = 0, hi = nb;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (bin_tile[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int32_t r = (i - bin_tile[lo]) * kAdTile;
    p.tiles[i] = make_int4(lo < L ? lo : -1, bin_row[lo] + r, min(kAdTile, tot[lo] - r), 0);
  }
  __syncthreads();  // bin_tile and bin_row end here
  const int lane = tid & 63, wave = tid >> 6;
  for (int base = r0; base < r1; base += kPlanThreads) {
    const int r = base + tid;
    const bool live = r < r1;
    if (base != r0) b = live ? bin_of(ids[r], L) : -1;
    if (nb <= kWaveBins) {
      for (int i = tid; i < W * nb; i += kPlanThreads) wcnt[i / nb][i % nb] = 0;
      __syncthreads();
    }
    uint64_t todo = __ballot(live), same = 0;
    while (todo) {
      const int lead = __builtin_ctzll(todo);
      const int lb = __builtin_amdgcn_readlane(b, lead);
      const uint64_t m = __ballot(live && b == lb);
      if (b == lb) same = m;
      todo &= ~m;
    }
    const int rank = __popcll(same & lanemask_lt());
    const int lead = same ? __builtin_ctzll(same) : 0;
    int32_t first = 0;
    if (nb <= kWaveBins) {
      if (live && lane == lead) wcnt[wave][b] = (uint16_t)__popcll(same);
      __syncthreads();
      for (int i = tid; i < nb; i += kPlanThreads) {  // counts to prefixes, in wave order
        uint32_t run = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t c = wcnt[w][i];
          wcnt[w][i] = (uint16_t)run;
          run += c;
        }
        tot[i] = next[i];       // where these rows of the bin begin
        next[i] += (int32_t)run;
      }
      __syncthreads();
      if (live) first = tot[b] + wcnt[wave][b];
      __syncthreads();          // both are written again in the next round
    } else {
      for (int w = 0; w < W; ++w) {
        if (wave == w && live && lane == lead) {
          first = next[b];
          next[b] = first + __popcll(same);
        }
        __syncthreads();
      }
      first = __shfl(first, lead, kWave);
    }
    if (live) p.order[first + rank] = r;
  }
}

// ------------------------------------------------------------------ low-rank values
// The vector memory unit takes the 16-byte accesses of four neighbouring lanes in
// one cycle where they are neighbours in memory, and in four where they are not (a
// matrix operand's neighbouring lanes are neighbouring ROWS: counted, 54 cache
// accesses per load instruction instead of 16, which bound the kernels). So a quad of
// lanes reads 64 contiguous bytes of one row per instruction, of its four rows in
// turn, and this turns the 4 x 4 pieces: in, register c of lane j is piece j of row c;
// out, register m of lane j is piece m of row j. Its own inverse.
template <int CTRL>
__device__ inline uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ inline void swap_pieces(uint4 &lo, uint4 &hi, bool upper) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t fb = dpp_u32<CTRL>(b[i]), fa = dpp_u32<CTRL>(a[i]);
    const uint32_t na = upper ? fb : a[i], nb = upper ? b[i] : fa;
    a[i] = na;
    b[i] = nb;
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}
__device__ inline void turn_quad(uint4 (&v)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  swap_pieces<0xB1>(v[0], v[1], odd);   // quad_perm [1,0,3,2]
  swap_pieces<0xB1>(v[2], v[3], odd);
  swap_pieces<0x4E>(v[0], v[2], high);  // quad_perm [2,3,0,1]
  swap_pieces<0x4E>(v[1], v[3], high);
}

// How the second product takes the low-rank values: `steps` matrix instructions of
// 32 places a row and 16 columns. The places hold the three bf16 parts of the
// scaled values: for rank 8 all three parts in one step (PACK 1), for rank 16 two
// and then the third (PACK 2), else 32 ranks of one part a step, the parts of a
// block of 32 ranks following each other (PACK 0). Other places hold zeros. In memory
// they lie as the instructions take them, [tile of 64 rows][16 rows][step][lane].
__host__ __device__ inline int part_pack(int rank) { return rank == 8 ? 1 : rank == 16 ? 2 : 0; }
__host__ __device__ inline int part_steps(int rank) { return rank <= 16 ? rank / 8 : 3 * ((rank + 31) / 32); }

// The low-rank values v of ranks 8 r8 .. of row i of a tile, where they go: low by
// row, and the scaled values' parts.
__device__ inline void put_low(const LowRankArgs &p, int tile, int i, int row, int r8, const float (&v)[8], float m) {
  const int pack = part_pack(p.rank), steps = part_steps(p.rank);
  float sv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sv[k] = v[k] * m;
  if (p.low && 8 * r8 < p.rank) store_elems8<false>(p.low, (int64_t)row * p.rank + 8 * r8, p.low_scaled ? sv : v);
  if (!p.parts) return;
  uint4 q[3];
  split3(sv, q[0], q[1], q[2]);
  uint4 *d = reinterpret_cast<uint4 *>(p.parts) + ((int64_t)tile * 4 + (i >> 4)) * steps * 64 + (i & 15);
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    const int g = pack == 1 ? part : 2 * part + r8;  // PACK 1 and 2: groups of 8 places one after the other
    const int step = pack ? g >> 2 : 3 * (r8 >> 2) + part, lane = 16 * (pack ? g & 3 : r8 & 3);
    d[step * 64 + lane] = q[part];
  }
  if (pack && r8 == 0)
    for (int g = 3 * pack; g < 4 * pack; ++g) d[(g >> 2) * 64 + 16 * (g & 3)] = make_uint4(0, 0, 0, 0);
}
// Groups of 8 ranks of a row, with the empty ones of the last block of 32.
__host__ __device__ inline int low_groups(int rank) { return part_pack(rank) ? rank / 8 : (rank + 31) / 32 * 4; }

// ------------------------------------------------------------------ shrink
// K is taken in slices, one workgroup per tile and slice, so that few rows still make
// many workgroups. Workgroups go to the 8 XCDs in turn, so with 2 or 4 slices a slice's
// workgroups share 4 or 2 XCDs, and its columns of a gathered x (each token's row is read
// by every expert that it was routed to) and of all adapters stay in those XCDs' L2; with
// 1 or 3 slices every XCD reads all columns.
// Inside, the W waves take every W-th 128-wide step of the slice for all the tile's
// rows, so each adapter row is read once per workgroup. A quad reads 64 bytes of one
// row, the four quads of a row 256. Four waves where there are many rows: eight take
// 31.4 us against 27.1 for 32768 gathered rows of rank 16, 89.7 against 57.1 of rank 64.
// Bound by the loads of x: 32768 contiguous rows of 2048 (134 MB) take 30 us, 4.5 TB/s,
// a plain read of them 24; 4096 rows gathered 8 times each 19.4 us, 6.9 TB/s out of L2.
constexpr int kSliceMin = 256;  // no slice is narrower

template <int RT, int NS, int W>
__device__ inline void shrink_rows(const LowRankArgs &p, const int32_t *order, int n, int l, int k, int k1, f32x4_t (&acc)[4][RT]) {
  const int lane = threadIdx.x & 63, q = lane >> 4, first = 4 * ((lane >> 2) & 3);  // this quad's rows: first + c
  int r[NS][4];
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int c = 0; c < 4; ++c) r[s][c] = order[min(16 * s + first + c, n - 1)];
  if (p.row_of) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) r[s][c] = p.row_of[r[s][c]];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) r[s][c] = min(max(r[s][c], 0), p.x_rows - 1);
  }
  const uint16_t *w0 = p.W1 + (int64_t)l * p.rank * p.K;
  for (; k < k1; k += 128 * W) {
    // Every load is made (places past the slice read its last ones, against zero
    // weights): no branch splits a step's loads.
    const int kl = k + 32 * q + 8 * (lane & 3), kc = min(kl, k1 - 8);
    // 16-rank blocks of weights in flight together: all 8 of rank 128 spill (8192 rows, 34.6 us against 31.8)
    constexpr int G = RT < 4 ? RT : 4;
    uint4 x[NS][4], w[G][4];
    auto load_w = [&](int j0) {
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) w[j][c] = load16(w0 + (int64_t)min(16 * (j0 + j) + first + c, p.rank - 1) * p.K + kc);
    };
    load_w(0);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[s][c] = load16(p.x + (int64_t)r[s][c] * p.K + kc);
#pragma unroll
    for (int j0 = 0; j0 < RT; j0 += G) {
      if (j0 > 0) load_w(j0);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (kl >= k1) w[j][0] = w[j][1] = w[j][2] = w[j][3] = make_uint4(0, 0, 0, 0);
        turn_quad(w[j]);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (j0 == 0) turn_quad(x[s]);
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[s][j0 + j] = mfma16(w[j][c], x[s][c], acc[s][j0 + j]);
      }
    }
  }
}

template <int RT, int W>
__global__ __launch_bounds__(64 * W) void k_shrink(LowRankArgs p, int slices, int slice) {
  constexpr int kPad = RT * 16 + 4, SL = RT <= 2 ? 4 : RT == 4 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float red[SL][kAdTile][kPad];
  const int si = blockIdx.x % slices, ti = blockIdx.x / slices;
  if (ti >= p.plan.counts[0]) return;
  const int4 tile = p.plan.tiles[ti];
  const int l = tile.x, n = tile.z, rank = p.rank;
  const int32_t *order = p.plan.order + tile.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int nr8 = rank / 8, g8 = low_groups(rank);
  if (l < 0) {  // rows without an adapter: low is 0, and the parts are not read
    if (slices == 1 && p.low)
      for (int i = tid; i < n * nr8; i += 64 * W) {
        const float z[8] = {};
        store_elems8<false>(p.low, (int64_t)order[i / nr8] * rank + 8 * (i % nr8), z);
      }
    return;
  }
  const int k = si * slice + 128 * wave, k1 = min(p.K, (si + 1) * slice);
  f32x4_t acc[4][RT] = {};
  if (n <= 16) shrink_rows<RT, 1, W>(p, order, n, l, k, k1, acc);
  else if (n <= 32) shrink_rows<RT, 2, W>(p, order, n, l, k, k1, acc);
  else shrink_rows<RT, 4, W>(p, order, n, l, k, k1, acc);
  // lane: row 16 s + l16, ranks 16 j + 4 q ..; the waves' sums in a fixed order, SL of them at a time
#pragma unroll
  for (int turn = 0; turn < W / SL; ++turn) {
    if (wave / SL == turn) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          f32x4_t *d = reinterpret_cast<f32x4_t *>(&red[wave % SL][16 * s + l16][16 * j + 4 * q]);
          *d = turn == 0 ? acc[s][j] : *d + acc[s][j];
        }
    }
    lds_barrier();
  }
  if (slices == 1) {  // nothing to join
    const float m = p.scale ? p.scale[l] : 1.0f;
    for (int i = tid; i < n * g8; i += 64 * W) {
      const int row = i / g8, r8 = i % g8;
      float v[8] = {};
      if (r8 < nr8) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float u = red[0][row][8 * r8 + c];
#pragma unroll
          for (int w = 1; w < SL; ++w) u += red[w][row][8 * r8 + c];
          v[c] = u;
        }
      }
      put_low(p, ti, row, order[row], r8, v, m);
    }
    return;
  }
  float *out = p.partial + ((int64_t)si * p.R + tile.y) * rank;
  const int r4 = rank / 4;
  for (int i = tid; i < n * r4; i += 64 * W) {
    f32x4_t v = *reinterpret_cast<const f32x4_t *>(&red[0][i / r4][4 * (i % r4)]);
#pragma unroll
    for (int w = 1; w < SL; ++w) v += *reinterpret_cast<const f32x4_t *>(&red[w][i / r4][4 * (i % r4)]);
    *reinterpret_cast<f32x4_t *>(out + 4 * i) = v;
  }
}

// The slices' sums, added in order, for 8 ranks of one row of a tile a thread.
__global__ __launch_bounds__(256) void k_shrink_join(LowRankArgs p, int slices) {
  const int nr8 = p.rank / 8, g8 = low_groups(p.rank);
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int ti = (int)(item / (kAdTile * g8)), i = (int)(item % (kAdTile * g8)) / g8, r8 = (int)(item % g8);
  if (ti >= p.plan.counts[0]) return;
  const int4 tile = p.plan.tiles[ti];
  if (i >= tile.z) return;
  const int l = tile.x, place = tile.y + i;
  float v[8] = {};
  if (l >= 0 && r8 < nr8) {
    for (int s = 0; s < slices; ++s) {
      float u[8];
      load_elems8<false>(p.partial, ((int64_t)s * p.R + place) * p.rank + 8 * r8, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += u[k];
    }
  }
  put_low(p, ti, i, p.plan.order[place], r8, v, p.scale && l >= 0 ? p.scale[l] : 1.0f);
}

// ------------------------------------------------------------------ expand
// A wave takes S blocks of 16 rows and 128 columns, a workgroup of four waves a tile
// of 64 rows and S x 128 columns; no LDS and no barrier. The product is taken
// transposed (columns as the matrix rows), so a lane ends with whole 16-byte pieces of
// one row's columns: pieces m = 0 .. 3 of the 128 (bf16) or twice 64 (fp32) columns,
// 4 q + m of 16. base comes and out goes by turn_quad, 256 contiguous bytes of a row
// per instruction, and the three meet in registers. Bound by HBM: 32768 x 2048 bf16 take
// 52 us, 5.2 TB/s. base and out pass by the caches, which hold what the next call reads:
// between the kernel that makes base and one that reads out, us for the three, 205 ->
// 201; 16384 x 2048 fp32 168 -> 158; 4099 x 5760 of rank 64 fp32 141 -> 133.
template <int PACK, bool BF, int S>
__global__ __launch_bounds__(256) void k_expand(LowRankArgs p, int blocks) {
  const int ti = blockIdx.x / blocks;  // a tile's column blocks follow each other: whole rows are in flight together
  if (ti >= p.plan.counts[0]) return;
  const int4 tile = p.plan.tiles[ti];
  const int l = tile.x, rank = p.rank, nr8 = rank / 8;
  if (l < 0 && p.base == p.out) return;  // nothing to add
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4, first = 4 * ((lane >> 2) & 3);
  constexpr int WR = 4 / S;  // waves along the rows; the others along the columns
  const int c0 = ((int)(blockIdx.x % blocks) * S + wave / WR) * 128, r0 = (wave % WR) * 16 * S;
  const int n = tile.z - r0;
  if (n <= 0 || c0 >= p.N) return;
  const int32_t *order = p.plan.order + tile.y + r0;
  int rows[S][4];  // this quad's rows: 16 s + first + c
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int c = 0; c < 4; ++c) rows[s][c] = order[min(16 * s + first + c, n - 1)];
  constexpr int NT = PACK ? PACK : 3, NB = BF ? 1 : 2, TPB = BF ? 8 : 4, E = BF ? 8 : 4;  // blocks, column tiles a block, values a piece
  const int steps = part_steps(rank);
  const uint4 *trow = reinterpret_cast<const uint4 *>(p.parts) + ((int64_t)ti * 4 + r0 / 16) * steps * 64 + lane;
  uint4 w[8], t[NT][S];
  auto load_t = [&](int o) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int s = 0; s < S; ++s) t[k][s] = trow[(s * steps + 3 * o + k) * 64];
  };
  // the weights of the ranks that this lane's 8 places of block o hold; places of no part meet zeros
  auto load_w = [&](int o) {
    const int r8 = PACK == 1 ? 0 : PACK == 2 ? (q & 1) : 4 * o + q;
    const bool ok = PACK == 1 ? q < 3 : PACK == 2 ? true : r8 < nr8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = BF ? 32 * (l16 >> 2) + 4 * j + (l16 & 3) : 64 * (j >> 2) + 16 * (l16 >> 2) + 4 * (j & 3) + (l16 & 3);
      const uint4 v = load16(p.W2 + ((int64_t)l * p.N + min(c0 + c, p.N - 1)) * rank + (ok ? 8 * r8 : 0));
      w[j] = ok ? v : make_uint4(0, 0, 0, 0);
    }
  };
  if (l >= 0) {
    load_w(0);
    load_t(0);
  }
  // base, in flight during the product (rows and columns past the end read the last
  // ones and are not stored)
  const int cq = c0 + 4 * E * q + E * (lane & 3);  // this lane's piece, of block 0
  uint4 base[S][NB][4];
  if (p.base) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t at = (int64_t)rows[s][c] * p.N + min(cq + 64 * b, p.N - E);
          base[s][b][c] = BF ? load16_nt(reinterpret_cast<const uint16_t *>(p.base) + at) : load16_nt(reinterpret_cast<const float *>(p.base) + at);
        }
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c) base[s][b][c] = make_uint4(0, 0, 0, 0);
  }
  f32x4_t acc[S][8] = {};  // [16 rows][16 columns]
  if (l >= 0) {
    if constexpr (PACK != 0) {
#pragma unroll
      for (int o = 0; o < PACK; ++o) {
        if (o == 1 && q >= 2) {  // the third part and 16 empty places; the other weights are the first step's
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[s][j] = mfma16(w[j], t[o][s], acc[s][j]);
      }
    } else {
      for (int o = 0; o < (nr8 + 3) / 4; ++o) {
        if (o > 0) {
          load_w(o);
          load_t(o);
        }
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[s][j] = mfma16(w[j], t[part][s], acc[s][j]);
      }
    }
  } else {  // base's bits: x + -0 is x, where x + 0 turns a -0 into 0
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[s][j] = {-0.0f, -0.0f, -0.0f, -0.0f};
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (16 * s >= n) break;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint4 (&v)[4] = base[s][b];
      turn_quad(v);  // pieces m = 0 .. 3 of row 16 s + l16
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if constexpr (BF) {
          float f[8];
          unpack_bf16x8(v[m], f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] += acc[s][2 * m][k];
            f[4 + k] += acc[s][2 * m + 1][k];
          }
          v[m] = pack_bf16x8(f);
        } else {
          const f32x4_t a = acc[s][TPB * b + m];
          v[m] = make_uint4(__float_as_uint(__uint_as_float(v[m].x) + a[0]), __float_as_uint(__uint_as_float(v[m].y) + a[1]),
                            __float_as_uint(__uint_as_float(v[m].z) + a[2]), __float_as_uint(__uint_as_float(v[m].w) + a[3]));
        }
      }
      turn_quad(v);
      const int c1 = cq + 64 * b;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (16 * s + first + c >= n || c1 >= p.N) continue;
        const int64_t at = (int64_t)rows[s][c] * p.N + c1;
        if constexpr (BF) store16_nt(reinterpret_cast<uint16_t *>(p.out) + at, v[c]);
        else store16_nt(reinterpret_cast<float *>(p.out) + at, v[c]);
      }
    }
  }
}

// ------------------------------------------------------------------ weight gradients
// Sums over rows: the contraction runs along the rows, across the storage order of
// both operands. A lane loads 8 neighbouring columns of 8 rows and turns the 8 x 8
// block in registers (one v_perm_b32 per pair of values), which gives it, for each
// of its 8 columns, 8 consecutive rows: the matrix operand, with no LDS. p's rows
// are split into three bf16 parts in registers. One workgroup per chunk of rows and
// 128 columns, its four waves taking every fourth step of 32 rows; their sums are
// added in order through LDS, from which they leave in either layout. An adapter
// with one chunk (of no rows: zeros), or so few that one workgroup takes all, is written
// straight out; the chunks of others go to partial sums that k_rowgrad_join adds in
// order. dA and dB run in one launch: dB waits for dy while dA, from an 8-bit x that the caches hold, decodes and turns; apart,
// one after the other, they take 64 us instead of 56 (32768 rows of rank 16, 2048 x
// 2048, dy 134 MB read once; vector instructions 20 us). Run right after the product
// that reads dy too, before the expansion: 49 us, the caches still hold a part of dy.
// Ranks above 64 take two workgroups along y, which read and turn dy and x twice: a whole
// backward of 32768 rows of rank 128 takes 378 us, of rank 64 224 (2048 x 2048). Above rank
// 32 an MXFP8 x needs 262 registers, one wave a SIMD instead of two: rank 64 262 us.
constexpr int kGradCols = 128;

template <int SRC, int RT>
__device__ inline void rowgrad_body(const RowGradOne &p, const int4 chunk, int cw, int j0, int rank, const int32_t *prow,
                                    const int32_t *vrow, float (*tile)[kGradCols + 4]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int l = chunk.x, n = chunk.z;
  const int c = min(cw + 8 * l16, p.C - 8);  // past the end: a valid place, not stored
  f32x4_t acc[RT][8] = {};
  for (int r0 = 32 * wave; r0 < n; r0 += 128) {
    uint32_t blk[4][8];  // rows (2 i, 2 i + 1) of column k as one word: [i][k]
    uint4 raw[8];
    uint32_t sc[8];
    const bool whole = r0 + 32 <= n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = (int64_t)vrow[min(r0 + 8 * q + i, n - 1)] * p.C + c;
      if constexpr (SRC == SRC_BF16) {
        raw[i] = load16(reinterpret_cast<const uint16_t *>(p.v) + at);
      } else {
        const uint2 w = load8(reinterpret_cast<const uint8_t *>(p.v) + at);
        raw[i] = make_uint4(w.x, w.y, 0, 0);
        sc[i] = p.v_scale[at >> 5];
      }
    }
    float pv[RT][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float *src = p.p + (int64_t)prow[min(r0 + 8 * q + i, n - 1)] * rank;
#pragma unroll
      for (int t = 0; t < RT; ++t) pv[t][i] = src[min(j0 + 16 * t + l16, rank - 1)];
    }
    if (!whole) {  // places past the chunk hold zeros in both operands (0 x infinity is not 0)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r0 + 8 * q + i >= n) {
          raw[i] = make_uint4(0, 0, 0, 0);
          sc[i] = 0;
#pragma unroll
          for (int t = 0; t < RT; ++t) pv[t][i] = 0.0f;
        }
    }
    uint4 a[RT][3];
#pragma unroll
    for (int t = 0; t < RT; ++t) split3(pv[t], a[t][0], a[t][1], a[t][2]);
    if constexpr (SRC == SRC_BF16) {
      turn_8x8(raw, blk);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int F = SRC - SRC_MXINT8;
        float x[8], y[8];
        ckpt8_decode8<F>(make_uint2(raw[2 * i].x, raw[2 * i].y), sc[2 * i], x);
        ckpt8_decode8<F>(make_uint2(raw[2 * i + 1].x, raw[2 * i + 1].y), sc[2 * i + 1], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) blk[i][k] = f32x2_to_bf16x2_rne(x[k], y[k]);  // exact
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 b = make_uint4(blk[0][k], blk[1][k], blk[2][k], blk[3][k]);
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int part = 0; part < 3; ++part) acc[t][k] = mfma16(a[t][part], b, acc[t][k]);
    }
  }
  // lane: columns cw + 8 l16 + k, ranks j0 + 16 t + 4 q ..
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float *d = &tile[16 * t + 4 * q + i][8 * l16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4_t v = {acc[t][4 * h][i], acc[t][4 * h + 1][i], acc[t][4 * h + 2][i], acc[t][4 * h + 3][i]};
            f32x4_t *e = reinterpret_cast<f32x4_t *>(d + 4 * h);
            *e = w == 0 ? v : *e + v;
          }
        }
    }
    lds_barrier();
  }
  const int64_t size = (int64_t)rank * p.C;
  float *out = chunk.w < 0 ? p.out + l * size : p.partial + chunk.w * size;
  const float m = p.scale && n > 0 ? p.scale[l] : 1.0f;  // no rows: zeros, whatever an unused slot's scale holds
  const int cols = min(kGradCols, p.C - cw), ranks = min(16 * RT, rank - j0);  // multiples of 8
  if (p.transposed) {
    const int r4 = ranks / 4;
    for (int i = tid; i < cols * r4; i += 256) {
      const int cc = i / r4, j = 4 * (i % r4);
      const f32x4_t v = {tile[j][cc], tile[j + 1][cc], tile[j + 2][cc], tile[j + 3][cc]};
      *reinterpret_cast<f32x4_t *>(out + (int64_t)(cw + cc) * rank + j0 + j) = v * m;
    }
  } else {
    const int c4 = cols / 4;
    for (int i = tid; i < ranks * c4; i += 256) {
      const int j = i / c4, cc = 4 * (i % c4);
      *reinterpret_cast<f32x4_t *>(out + (int64_t)(j0 + j) * p.C + cw + cc) = *reinterpret_cast<const f32x4_t *>(&tile[j][cc]) * m;
    }
  }
}

template <int SRC, int RT>
__global__ __launch_bounds__(256) void k_rowgrad(RowGradArgs p, int na, int nb) {
  __shared__ __attribute__((aligned(16))) float tile[16 * RT][kGradCols + 4];
  __shared__ int32_t prow[kMaxChunk], vrow[kMaxChunk];
  const int per = na + nb, ci = blockIdx.x / per, block = blockIdx.x % per;
  if (ci >= p.plan.counts[1]) return;
  int4 chunk = p.plan.chunks[ci];
  if (p.merge > 1 && chunk.w >= 0) {  // the first of `merge` chunks takes them all
    const int2 of = p.plan.chunks_of[chunk.x];
    const int k = chunk.w - of.y;
    if (k % p.merge) return;
    const int4 end = p.plan.chunks[ci + min(p.merge, of.x - k) - 1];
    chunk.z = end.y + end.z - chunk.y;
    if (of.x <= p.merge) chunk.w = -1;
  }
  const bool first = block < na;
  const int32_t *row_of = first ? p.a.row_of : p.b.row_of;
  const int last = (first ? p.a.v_rows : p.b.v_rows) - 1;
  for (int i = threadIdx.x; i < chunk.z; i += 256) {
    const int r = p.plan.order[chunk.y + i];
    prow[i] = r;
    vrow[i] = row_of ? min(max(row_of[r], 0), last) : r;
  }
  lds_barrier();
  const int j0 = blockIdx.y * (16 * RT);
  if (first) rowgrad_body<SRC, RT>(p.a, chunk, block * kGradCols, j0, p.rank, prow, vrow, tile);
  else rowgrad_body<SRC_BF16, RT>(p.b, chunk, (block - na) * kGradCols, j0, p.rank, prow, vrow, tile);
}

// The chunks of an adapter that has several, added in order.
__global__ __launch_bounds__(256) void k_rowgrad_join(RowGradArgs p, int64_t sa, int64_t sb) {
  const int2 c = p.plan.chunks_of[blockIdx.y];
  if (c.x <= p.merge) return;
  int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= sa + sb) return;
  const bool first = i < sa;
  const int64_t size = first ? sa : sb;
  if (!first) i -= sa;
  const float *partial = (first ? p.a.partial : p.b.partial) + c.y * size + i;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < c.x; k += p.merge) s += *reinterpret_cast<const f32x4_t *>(partial + k * size);
  *reinterpret_cast<f32x4_t *>((first ? p.a.out : p.b.out) + blockIdx.y * size + i) = s;
}

__global__ __launch_bounds__(256) void k_zero_f32(float *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// ------------------------------------------------------------------ few rows
// One launch, no plan: a workgroup per row and share of the columns. Its W waves
// take the ranks in turn (a dot product over K each, two at a time), then every
// thread its columns. The workgroups of a row repeat its first product: A_l comes
// from L2 after the first, and a second launch would cost more. Bound by the latency of
// the two dependent products: 64 rows of rank 16 on 2048 x 2048 take 4 us, and a call
// 11, most of it the host's.
template <bool BF, int W>
__global__ __launch_bounds__(64 * W) void k_adapter_rows(AdapterRowsArgs p, int csplit) {
  __shared__ float ts[kMaxRank];
  const int r = blockIdx.x / csplit, cs = blockIdx.x % csplit, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = p.ids[r], rank = p.rank;
  const bool has = l >= 0 && l < p.L;
  if (has) {
    int xr = r;
    if (p.row_of) xr = min(max(p.row_of[r], 0), p.x_rows - 1);
    const uint16_t *x = p.x + (int64_t)xr * p.K;
    const uint16_t *A = p.A + (int64_t)l * rank * p.K;
    for (int j = wave; j < rank; j += 2 * W) {  // ranks j and j + W
      const int j1 = min(j + W, rank - 1);
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
      for (int k = 8 * lane; k < p.K; k += 512) {
        float xv[8], a0[8], a1[8];
        load_elems8<true>(x, k, xv);
        load_elems8<true>(A, (int64_t)j * p.K + k, a0);
        load_elems8<true>(A, (int64_t)j1 * p.K + k, a1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s0 += xv[i] * a0[i];
          s1 += xv[i] * a1[i];
        }
      }
      s0 = wave_sum(s0);
      s1 = wave_sum(s1);
      if (lane == 0) {
        ts[j] = s0;
        if (j + W < rank) ts[j + W] = s1;
      }
    }
  }
  lds_barrier();
  if (p.t && cs == 0)
    for (int j = tid; j < rank; j += 64 * W) p.t[(int64_t)r * rank + j] = has ? ts[j] : 0.0f;
  const float m = has && p.scale ? p.scale[l] : 1.0f;
  const int blocks = (p.N + 255) / 256;
  const int c1 = min(p.N, 256 * (int)((int64_t)blocks * (cs + 1) / csplit));
  for (int c = 256 * (int)((int64_t)blocks * cs / csplit) + tid; c < c1; c += 64 * W) {
    const int64_t at = (int64_t)r * p.N + c;
    float b = 0.0f;
    if (p.base) b = BF ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p.base)[at]) : reinterpret_cast<const float *>(p.base)[at];
    if (has) {
      const uint16_t *w = p.B + ((int64_t)l * p.N + c) * rank;
      float s = 0.0f;
#pragma unroll 2
      for (int j = 0; j < rank; j += 8) {
        float v[8];
        load_elems8<true>(w, j, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i] * ts[j + i];
      }
      b += m * s;
    }
    if (BF) reinterpret_cast<uint16_t *>(p.out)[at] = (uint16_t)f32_to_bf16_rne(b);
    else reinterpret_cast<float *>(p.out)[at] = b;
  }
}

}  // namespace

// Rows of a gradient chunk: about 32 chunks' worth of rows, 128 to kMaxChunk.
int adapter_chunk_rows(int R) {
  const int64_t c = cdiv(cdiv(R, 32), 64) * 64;
  return (int)(c < 128 ? 128 : c > kMaxChunk ? kMaxChunk : c);
}

size_t adapter_plan_layout(int R, int L, void *base, AdapterPlan *p) {
  const int bins = R < L + 1 ? R : L + 1;
  const int64_t ch = adapter_chunk_rows(R);
  AdapterPlan q;
  q.max_tiles = (int)cdiv(R, kAdTile) + bins;
  q.max_chunks = (int)cdiv(R, ch) + L;
  // an adapter of n > 1 chunks has more than (n - 1) ch rows, so n <= 2 rows / ch
  q.max_slots = (int)(2 * cdiv(R, ch));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char *at = base ? (char *)base + off : nullptr;
    off = align_up(off + bytes);
    return (void *)at;
  };
  q.order = (int32_t *)take(sizeof(int32_t) * (size_t)R);
  q.counts = (int32_t *)take(sizeof(int32_t) * 2);
  q.chunks_of = (int2 *)take(sizeof(int2) * (size_t)L);
  q.tiles = (int4 *)take(sizeof(int4) * (size_t)q.max_tiles);
  q.chunks = (int4 *)take(sizeof(int4) * (size_t)q.max_chunks);
  q.hist = (int32_t *)take(sizeof(int32_t) * (size_t)cdiv(R, plan_rows(R, L)) * (L + 1));
  if (p) *p = q;
  return off;
}

hipError_t launch_adapter_prepare(const PrepareArgs &a, hipStream_t s) {
  const int per = plan_rows(a.R, a.L);
  const int groups = a.ids ? (int)cdiv(a.R, per) : 0;
  const bool self = a.R <= kSelfCount;
  const int threads = groups ? kPlanThreads : kPrepareThreads;  // the weights are turned beside the grouping, or alone
  const TurnPair turn = {{a.B, a.Bt, a.N, a.rank, false}, {a.A, a.At, a.rank, a.K, true},
                         a.Bt ? (int)cdiv((int64_t)a.N * a.rank / 64, threads) : 0,
                         a.At ? (int)cdiv((int64_t)a.K * a.rank / 64, threads) : 0};
  const unsigned turns = (unsigned)(a.L * (turn.b0 + turn.b1));
  if (groups == 0 && turns > 0) hipLaunchKernelGGL(k_turn, dim3(turns), dim3(kPrepareThreads), 0, s, turn);
  if (groups == 0) return hipGetLastError();
  if (!self)
    hipLaunchKernelGGL(k_plan_hist, dim3(groups), dim3(kPrepareThreads), sizeof(int32_t) * (a.L + 1), s, a.ids, a.R, a.L, per,
                       a.plan.hist);
  hipLaunchKernelGGL(k_plan_scatter, dim3(groups + turns), dim3(kPlanThreads), 0, s, a.ids, a.R, a.L, per, groups, self,
                     adapter_chunk_rows(a.R), a.plan, turn);
  return hipGetLastError();
}

// Slices of K, each a multiple of 128 and at least kSliceMin wide: up to 4, as many as
// make no more workgroups of 64 rows than there are CUs; where one slice already makes
// more (from 16384 rows), 4 for ranks up to 16 and 2 above. Ranks above 32 hold one
// workgroup a CU (their registers); lower ones two or three, and take the same rule.
// The rule is not the fastest everywhere: from 16384 rows of rank 64, 1 slice was 4 us
// faster than its 2 at K = 2048 and 4 slices 4 us faster at K = 4096. us, product +
// join, for 1 / 2 / 3 / 4 / 8:
//   640 rows, rank 32, K 4096       19.6 / 16.3 /      / 12.7 / 11.6
//   2000 rows, rank 64, K 2880           / 18.1 / 16.6 / 15.1
//   4099 rows, rank 64, K 2880      22.5 / 19.4 / 18.1 / 23.2 / 24.4
//   6500 rows, rank 64, K 2880           / 19.6 / 26.0 / 24.3
//   8192 rows, rank 16, K 2048      13.4 / 16.6 /      / 16.6 / 17.5
//   12867 rows, rank 64, K 1568     19.6 / 26.9 /      / 33.2 / 40.6
//   16384 rows, rank 64, K 4096     67.1 / 63.7 /      / 59.7 / 71.2
//   32768 rows, rank 64, K 2048     57.1 / 61.2 /      / 72.4 / 114
//   32768 rows, rank 16, K 2048     44.1 / 42.0 /      / 40.3 / 43.3
// Few rows of a low rank take one slice with 8 waves a workgroup, without a join,
// while K is not too long for it (640 rows, rank 32, K 4096 17.0 us, 2048 rows, rank 16
// 13.8): 1003 rows, rank 32, K 1440 10.3 us against 6.2 + 5.1 and a launch, a backward
// of 168 rows, rank 16, 2784 x 2744 40 us against 43.
static bool deep_slice(int R, int K, int rank) { return R < 4096 && rank <= 32 && K > 512 && K < 3000; }
static int slice_width(int R, int K, int rank) {
  const int fit = (256 * kAdTile - 1) / R;  // an adapter more makes a tile more
  const int most = fit > 0 ? (fit < 4 ? fit : 4) : rank <= 16 ? 4 : 2;
  const int w = (int)cdiv(cdiv(K, K <= 512 || deep_slice(R, K, rank) ? 1 : most), 128) * 128;
  return w < kSliceMin ? kSliceMin : w;
}
int adapter_slices(int R, int K, int rank) { return (int)cdiv(K, slice_width(R, K, rank)); }
size_t adapter_parts_elems(int tiles, int rank) { return (size_t)tiles * kAdTile * 32 * part_steps(rank); }

template <int PACK, int S>
static void expand_one(const LowRankArgs &a, hipStream_t s) {
  const int blocks = (int)cdiv(a.N, 128 * S);
  const dim3 grid((unsigned)(a.plan.max_tiles * blocks));
  if (a.bf16) hipLaunchKernelGGL((k_expand<PACK, true, S>), grid, dim3(256), 0, s, a, blocks);
  else hipLaunchKernelGGL((k_expand<PACK, false, S>), grid, dim3(256), 0, s, a, blocks);
}

hipError_t launch_adapter_shrink(const LowRankArgs &a, hipStream_t s) {
  const int slice = slice_width(a.R, a.K, a.rank), slices = adapter_slices(a.R, a.K, a.rank);
  const dim3 grid((unsigned)(a.plan.max_tiles * slices)), block(256);
  const bool deep = deep_slice(a.R, a.K, a.rank);
  if (a.rank <= 16 && deep) hipLaunchKernelGGL((k_shrink<1, 8>), grid, dim3(512), 0, s, a, slices, slice);
  else if (a.rank <= 16) hipLaunchKernelGGL((k_shrink<1, 4>), grid, block, 0, s, a, slices, slice);
  else if (a.rank <= 32 && deep) hipLaunchKernelGGL((k_shrink<2, 8>), grid, dim3(512), 0, s, a, slices, slice);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_shrink<2, 4>), grid, block, 0, s, a, slices, slice);
  else if (a.rank <= 64) hipLaunchKernelGGL((k_shrink<4, 4>), grid, block, 0, s, a, slices, slice);
  else hipLaunchKernelGGL((k_shrink<8, 4>), grid, block, 0, s, a, slices, slice);
  if (slices > 1) {
    const int64_t items = (int64_t)a.plan.max_tiles * kAdTile * low_groups(a.rank);
    hipLaunchKernelGGL(k_shrink_join, dim3((unsigned)cdiv(items, 256)), block, 0, s, a, slices);
  }
  return hipGetLastError();
}

hipError_t launch_adapter_expand(const LowRankArgs &a, hipStream_t s) {
  const int pack = part_pack(a.rank);
  // Two blocks of 16 rows a wave for a high rank, whose weights are then read half as
  // often, unless the workgroups get few. us, one block against two: rank 128, 8192
  // rows, N = 4096 91.8 / 79.6; rank 64, 12867 rows, N = 2048 47.2 / 42.4, 2048 rows
  // 12.0 / 11.8; rank 32, 8192 rows 17.9 / 18.9; rank 16, 32768 rows 52.2 / 53.9. (4096 rows
  // lie between the measured 2048, where both are even, and 8192.)
  if (pack == 1) expand_one<1, 1>(a, s);
  else if (pack == 2) expand_one<2, 1>(a, s);
  else if (a.rank > 32 && a.R >= 4096) expand_one<0, 2>(a, s);
  else expand_one<0, 1>(a, s);
  return hipGetLastError();
}

template <int SRC>
static void rowgrad_src(const RowGradArgs &a, hipStream_t s) {
  const dim3 block(256);
  const int na = a.a.out ? (int)cdiv(a.a.C, kGradCols) : 0, nb = a.b.out ? (int)cdiv(a.b.C, kGradCols) : 0;
  const unsigned gx = (unsigned)((int64_t)a.plan.max_chunks * (na + nb));
  if (a.rank <= 16) hipLaunchKernelGGL((k_rowgrad<SRC, 1>), dim3(gx), block, 0, s, a, na, nb);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_rowgrad<SRC, 2>), dim3(gx), block, 0, s, a, na, nb);
  else hipLaunchKernelGGL((k_rowgrad<SRC, 4>), dim3(gx, (unsigned)cdiv(a.rank, 64)), block, 0, s, a, na, nb);
}

hipError_t launch_adapter_rowgrad(const RowGradArgs &args, hipStream_t s) {
  // A chunk's partial sums are rank x 128 fp32 a workgroup, as many bytes as its rows of
  // a high rank: then more chunks to a workgroup, and where all of them fit no join. us, dA
  // and dB with the join, for 1 / 2 / 4 / 8 chunks:
  //   1003 rows of 5 adapters, 2880 x 1440, rank 16   9.9 / 9.0 / 8.9 / 7.5, rank 128 31.7 / 22.4 / 22.5 / 18.3
  //   4096 rows of 8, 2048 x 2048, rank 16 16.7 / 17.1 / 17.5 / 17.5, 32 24.3 / 20.2 / 21.8 / 21.3,
  //                                rank 64 44.1 / 35.3 / 28.6 / 29.9, 128 73.3 / 55.8 / 46.2 / 33.7
  //   12288 rows of 8, rank 32 37.0 / 36.5 / 49.3 / 43.5, 64 60.9 / 52.0 / 57.4 / 56.7, 128 108 / 92.7 / 83.5 / 90.3
  //   32768 rows of 4 (chunks of 1024), rank 32 71.0 / 74.9, 64 101.5 / 90.9, 128 193 / 172
  // 4 chunks above rank 32 is one number for all of these: 4096 rows of rank 128 would take
  // 8 (33.7 against 46.2), 12288 of rank 64 2 (52.0 against 57.4).
  RowGradArgs a = args;
  const int rows = adapter_chunk_rows(a.R);
  a.merge = a.R <= 8 * rows ? 8 : a.rank <= 16 ? 1 : a.rank <= 32 ? (a.R < 8192 ? 2 : 1) : 4;
  while (a.merge * rows > kMaxChunk) a.merge /= 2;
  if (a.src == SRC_BF16) rowgrad_src<SRC_BF16>(a, s);
  else if (a.src == SRC_MXINT8) rowgrad_src<SRC_MXINT8>(a, s);
  else rowgrad_src<SRC_MXFP8>(a, s);
  const int64_t sa = a.a.out ? (int64_t)a.rank * a.a.C : 0, sb = a.b.out ? (int64_t)a.rank * a.b.C : 0;  // multiples of 64
  if (a.R > a.merge * rows)  // else no adapter has partial sums
    hipLaunchKernelGGL(k_rowgrad_join, dim3((unsigned)cdiv(sa + sb, 1024), (unsigned)a.L), dim3(256), 0, s, a, sa, sb);
  return hipGetLastError();
}

hipError_t launch_fill_f32_zero(float *p, int64_t n, hipStream_t s) {
  const int64_t g = cdiv(n, 256);
  hipLaunchKernelGGL(k_zero_f32, dim3((unsigned)(g < 4096 ? g : 4096)), dim3(256), 0, s, p, n);
  return hipGetLastError();
}

// Shares of a row's columns in the one-launch form: until there are two workgroups
// per CU, and no fewer than 256 columns each.
static int rows_csplit(int R, int N) {
  const int64_t most = cdiv(N, 256), want = cdiv(512, R);
  return (int)(want < most ? want : most);
}

// Where the one-launch form runs: while at most 1 MB of A and B passes through one
// CU. Both forms, a pass in us on K = N = 2048: rank 16, 1024 / 2048 rows 14 / 23
// against 23 / 27 for the grouped kernels; rank 64, 256 / 512 rows 21 / 29 against 25
// / 27; and 2880 x 2880, rank 32: 256 / 1024 rows 17 / 29 against 22 / 27. (512 rows of
// rank 64 lie on the limit and still run here, 2 us behind.)
bool adapter_rows_supported(int R, int K, int N, int rank) {
  const int cs = rows_csplit(R, N);
  const int64_t bytes = cdiv((int64_t)R * cs, 256) * 2 * rank * ((int64_t)K + cdiv(N, cs));  // of A and B through one CU
  return bytes <= 1 << 20;
}

hipError_t launch_adapter_rows(const AdapterRowsArgs &a, hipStream_t s) {
  const int cs = rows_csplit(a.R, a.N);
  const dim3 grid((unsigned)(a.R * cs));
  // 16 waves where a CU has no second workgroup anyway and the ranks feed them
  if (a.R * cs <= 256 && a.rank >= 32) {
    if (a.bf16) hipLaunchKernelGGL((k_adapter_rows<true, 16>), grid, dim3(1024), 0, s, a, cs);
    else hipLaunchKernelGGL((k_adapter_rows<false, 16>), grid, dim3(1024), 0, s, a, cs);
  } else {
    if (a.bf16) hipLaunchKernelGGL((k_adapter_rows<true, 4>), grid, dim3(256), 0, s, a, cs);
    else hipLaunchKernelGGL((k_adapter_rows<false, 4>), grid, dim3(256), 0, s, a, cs);
  }
  return hipGetLastError();
}

}  // namespace nf4moe
