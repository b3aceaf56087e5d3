// Tiled bf16 product of the weight-only operators on many rows (gfx950):
//
//   C[m, b] = sum_r A[m, r] B[b, r]      (fp32 sums)
//
// A in one or two segments along r (A0, A1 [M, width], the columns of one after
// the other's), B the weights in bf16 as the dequantizing kernels lay them out:
// for every 256 rows b and every 32 r a block of 16 KB [256][32], each segment
// padded with zeros to whole chunks of 64 (so a tile's stage is read from
// consecutive addresses, whatever the row length: 8% of the time of a 24576-long
// reduction, where rows are multiples of 4 KB apart).
//
// 256 x 256 tiles, 8 waves of 128 x 64 on v_mfma_f32_32x32x16_bf16, both operands
// brought to LDS by the load unit (global_load_lds, 16 bytes a lane) in stages of
// 32 r, through a ring of NST buffers: NST - 1 stages are on their way while one is
// used.  LDS reads and transfers are issued one at a time between the MFMAs, which
// gave 7% over the same ring with the reads in front of them: the eight waves
// leave a barrier together and queue for LDS together.
//
// Measured, 4096 rows: 4096 -> 2 x 12288 columns 640-675 us (1.2-1.3 PFLOP/s),
// 24576 -> 4096 columns 606-640 us.  The matrix units are busy 74-79% of the cycles
// and the clock falls to 1.6 GHz: power bounds it, so a schedule with fewer idle
// cycles gains less than the cycles it saves.  (torch's library product of the same
// shapes takes 645 and 573 us.)
//
// LDS rows are 64 bytes, 4 slots of 16; slot s of row r holds piece
// s ^ ((r >> 2) & 3), so that the 16 lanes of one ds_read_b128 phase (rows
// r..r+15, one piece) touch 16 different groups of 4 banks.  The load unit writes a
// wave's 64 pieces consecutively, so the permutation is applied to the global
// addresses.
#pragma once

#include "w4a16.h"

#include <type_traits>

namespace svdq_gemm {

using namespace svdq_dev;

constexpr int BM = 256, BN = 256;
constexpr int NT = 512;
constexpr int WM = 128, WN = 64;
constexpr int RBL = WM / 32, CBL = WN / 32;

constexpr int BLOCK_BYTES = BN * 64;     // of B: 256 rows, 32 r

// bytes of B for `rows` rows and `stages` stages of 32 r
inline size_t weight_bytes(int64_t rows, int64_t stages) {
  return size_t((rows + BN - 1) / BN) * size_t(stages) * BLOCK_BYTES;
}

// where element (row, r) of B lies, r a multiple of 8
__device__ __forceinline__ uint4* weight_at(uint16_t* B, int64_t stages, int64_t row, int64_t r) {
  return reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(B) +
                                  ((row / BN) * stages + r / 32) * BLOCK_BYTES +
                                  (row % BN) * 64 + (r % 32) * 2);
}

struct Args {
  const uint16_t* A[2];
  int64_t width;          // columns of A in one segment (a multiple of 8)
  int chunks;             // chunks of 64 in one segment
  int segments;           // 1 or 2
  const uint16_t* B;
  int M, rows;            // rows of A, rows of B
};

constexpr int NST = 5;                   // stages in LDS, 32 KB each

struct __attribute__((aligned(16))) Stage {
  uint4 a[BM * 4];
  uint4 b[BN * 4];
};

// The epilogues use the stages' LDS again: each wave FLOATS consecutive floats inside
// one Stage (the stages are separate objects, in no promised order, and the compiler
// takes a pointer into one as apart from the others).  Which of st0, st1, st2 and
// at which float of it:
constexpr int EPILOGUE_STAGES = 3;

constexpr int epilogue_stage(int floats, int wave) { return wave / (int(sizeof(Stage)) / (4 * floats)); }

constexpr int epilogue_offset(int floats, int wave) {
  return wave % (int(sizeof(Stage)) / (4 * floats)) * floats;
}

template <int FLOATS>
__device__ __forceinline__ float* epilogue_buffer(int wave, Stage& st0, Stage& st1, Stage& st2) {
  static_assert(FLOATS % 4 == 0 && epilogue_stage(FLOATS, NT / 64 - 1) < EPILOGUE_STAGES,
                "the waves' buffers fit the stages");
  const int s = epilogue_stage(FLOATS, wave);
  return reinterpret_cast<float*>(s == 0 ? &st0 : s == 1 ? &st1 : &st2) +
         epilogue_offset(FLOATS, wave);
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// acc += the tile at (m0, b0), b0 a row of B.  All 512 threads call it.  The
// stages are separate LDS objects, so that the compiler can tell the one a
// transfer fills apart from the ones that are read.  `count` stages from `first` on (0:
// all of them).
__device__ __forceinline__ void tile_product(const Args& p, int64_t m0, int64_t b0, Stage& st0,
                                             Stage& st1, Stage& st2, Stage& st3, Stage& st4,
                                             v16f (&acc)[RBL][CBL], int first = 0, int count = 0) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int h = lane >> 5, r32 = lane & 31;

  // Wave w brings rows 32 w .. 32 w + 31 of both operands, 16 rows to a
  // transfer.  Rows past the edge repeat the last row (their products reach
  // only outputs that are never stored); pieces past A's width repeat its
  // last piece (the weights there are zeros).
  // The addresses are a uniform base and a lane's 32-bit offset in bytes (rows
  // and widths are at most 2^22 elements), which costs no vector instruction.
  const uint32_t piece = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
  uint32_t aoff[2], boff[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r = 32 * wave + 16 * t + (lane >> 2);
    aoff[t] = 2 * uint32_t(min(int64_t(r), p.M - 1 - m0)) * uint32_t(p.width);
    boff[t] = 64 * uint32_t(min(int64_t(r), p.rows - 1 - b0)) + piece;
  }
  const int seg = 2 * p.chunks, all = seg * p.segments, total = count ? count : all;
  const uint8_t* const a0 = reinterpret_cast<const uint8_t*>(p.A[0] + m0 * p.width);
  const uint8_t* const a1 = reinterpret_cast<const uint8_t*>(p.A[1] + m0 * p.width);
  const uint8_t* const bb =
      reinterpret_cast<const uint8_t*>(p.B) + b0 / BN * all * int64_t(BLOCK_BYTES);
  // transfer t of stage s: 0, 1 of A, 2, 3 of B
  const uint8_t *asrc, *bsrc;
  uint32_t apiece;
  auto dma_at = [&](int s) __attribute__((always_inline)) {
    s = first + min(s, total - 1);
    const bool second = s >= seg;
    // pieces that would lie past A's width repeat its last one
    const int col = min(32 * (second ? s - seg : s), int(p.width) - 8);
    apiece = min(piece, 2 * uint32_t(int(p.width) - 8 - col));
    asrc = (second ? a1 : a0) + 2 * col;
    bsrc = bb + BLOCK_BYTES * int64_t(s);
  };
  auto dma = [&](int t, Stage& st) __attribute__((always_inline)) {
    if (t < 2)
      __builtin_amdgcn_global_load_lds(asrc + (aoff[t & 1] + apiece),
                                       (lds_ptr_t)&st.a[(32 * wave + 16 * (t & 1)) * 4], 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds(bsrc + boff[t & 1],
                                       (lds_ptr_t)&st.b[(32 * wave + 16 * (t & 1)) * 4], 16, 0, 0);
  };

  const int sw = h ^ ((r32 >> 2) & 3);
  const int abase = (wm * WM + r32) * 4, bbase = (wn * WN + r32) * 4;
  v8bf fa[2][RBL], fb[2][CBL];
  // fragment n of half ks, in the order in which the MFMAs need them
  auto frag = [&](const Stage& st, int ks, int n) __attribute__((always_inline)) {
    const int slot = sw ^ (2 * ks);
    if (n == 0 || n == 2)
      fb[ks][n / 2] = __builtin_bit_cast(v8bf, st.b[bbase + 64 * n + slot]);
    else
      fa[ks][n == 1 ? 0 : n - 2] =
          __builtin_bit_cast(v8bf, st.a[abase + 128 * (n == 1 ? 0 : n - 2) + slot]);
  };
  auto mfma = [&](int ks, int n) __attribute__((always_inline)) {
    const int i = n / CBL, j = n % CBL;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[ks][i], fb[ks][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // One stage.  Its first half's fragments are in registers (or on their way).
  // LDS reads and transfers go out one at a time between MFMAs: issued in a row
  // they would hold the matrix core up, since the eight waves queue for LDS
  // together.  After the first half every wave waits for its own transfers of
  // the next stage (the NST - 2 stages after that may stay in flight) and for
  // its LDS reads; past the barrier the next stage is complete, this one's
  // buffer is free and is filled again, and the next stage's first fragments are
  // read.  Past the last stage the transfers repeat it.
  auto step = [&](int s, Stage& cur, Stage& nxt) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      mfma(0, n);
      if (n < 6) frag(cur, 1, n);
      if (n == 6) dma_at(s + NST);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0x0070 | (4 * (NST - 2)));   // vmcnt(4 (NST - 2)) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      mfma(1, n);
      if (n < 6) frag(nxt, 0, n);
      if (n & 1) dma(n / 2, cur);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(NST == 5, "the unrolled ring");
  auto fill = [&](int s, Stage& st) __attribute__((always_inline)) {
    dma_at(s);
#pragma unroll
    for (int t = 0; t < 4; ++t) dma(t, st);
  };
  fill(0, st0);
  fill(1, st1);
  fill(2, st2);
  fill(3, st3);
  fill(4, st4);
  // vmcnt(4 (NST - 1)): its low four bits and, at bit 14, its high two
  __builtin_amdgcn_s_waitcnt(0x0F70 | ((4 * (NST - 1)) & 15) | ((4 * (NST - 1)) >> 4 << 14));
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int n = 0; n < 6; ++n) frag(st0, 0, n);
  int s = 0;
  for (; s + NST <= total; s += NST) {
    step(s, st0, st1);
    step(s + 1, st1, st2);
    step(s + 2, st2, st3);
    step(s + 3, st3, st4);
    step(s + 4, st4, st0);
  }
  if (s < total) step(s, st0, st1);
  if (s + 1 < total) step(s + 1, st1, st2);
  if (s + 2 < total) step(s + 2, st2, st3);
  if (s + 3 < total) step(s + 3, st3, st4);
  // the repeated last transfers, before the buffers are used for anything else
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
}

// Tiles whose number is no multiple of the 256 compute units leave a last round that is
// partly empty.  Where that is most of the chip, the last round's tiles are split over
// the reduction as well: the first `full` workgroups take whole tiles, then S workgroups
// take a tile of the `left` others each, into fp32 sums [left][S][256][256] that a launch
// of its own joins.  4608 rows 4096 -> 12288 are 864 tiles, 3.4 rounds.
struct Rounds {
  int64_t full, left;
  int S;                  // 1: nothing is split
};

constexpr int64_t UNITS = 256;
constexpr int64_t TILE = int64_t(BM) * BN;

inline Rounds rounds(int64_t M, int64_t rows, int64_t stages) {
  const int64_t tiles = (M + BM - 1) / BM * ((rows + BN - 1) / BN);
  Rounds r{tiles / UNITS * UNITS, tiles % UNITS, 1};
  if (r.left) r.S = int(std::min<int64_t>({UNITS / r.left, 8, stages / 16}));
  if (r.S <= 1) r = {tiles, 0, 1};
  return r;
}

inline size_t rounds_bytes(const Rounds& r) { return size_t(r.left) * size_t(r.S) * TILE * 4; }

// this workgroup's tile; of a split one also its number among them and its stages
struct Work {
  int64_t m0, b0;
  int split, first, count;       // split -1: a whole tile
};

__device__ __forceinline__ void tile_of(int64_t t, int tiles_m, int tiles_n, int64_t& m0,
                                        int64_t& b0) {
  constexpr int GN = 8;
  const int grp = int(t / (GN * tiles_m)), in = int(t - int64_t(grp) * (GN * tiles_m));
  const int gn = min(GN, tiles_n - grp * GN);
  m0 = int64_t(in / gn) * BM;
  b0 = int64_t(grp * GN + in % gn) * BN;
}

__device__ __forceinline__ Work work_of(const Args& p, int64_t full, int S) {
  Work w;
  const int tm = (p.M + BM - 1) / BM, tn = (p.rows + BN - 1) / BN;
  const int64_t t = blockIdx.x;
  if (t < full) {
    // a run of whole tiles for each XCD
    tile_of((full & 7) == 0 ? (t & 7) * (full >> 3) + (t >> 3) : t, tm, tn, w.m0, w.b0);
    w.split = -1;
    w.first = w.count = 0;
    return w;
  }
  const int i = int(t - full), slice = i % S, stages = 2 * p.chunks;
  w.split = i / S;
  tile_of(full + w.split, tm, tn, w.m0, w.b0);
  w.first = int(int64_t(slice) * stages / S);
  w.count = int(int64_t(slice + 1) * stages / S) - w.first;
  w.split = i;
  return w;
}

template <int R, int C>
__device__ __forceinline__ void zero_acc(v16f (&acc)[R][C]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
}

}  // namespace svdq_gemm

// Measured: gated pair 333 rows 2048 -> 8208 40 us (0.56 PFLOP/s), 1000 rows
// 4096 -> 12288 225 us (0.90); a copy of the kernel without the dequantization took 29
// us at 333 rows: its vector instructions and the MFMAs add up on a SIMD instead of
// overlapping, and 387 tiles leave a quarter of the chip idle in the second half.
//
// A medium number of rows: 128 x 128 tiles, 4 waves of 64 x 64, two workgroups
// to a compute unit.  A comes to LDS by the load unit; the weights are
// dequantized on their way into LDS (once per 128 rows, where a pass of their
// own would cost more than it saves).  Few tiles are split over the reduction
// as well, into S slices of whole chunks.
namespace svdq_mid {

using namespace svdq_dev;
using svdq_gemm::lds_ptr_t;
using svdq_gemm::zero_acc;

constexpr int BM = 128, BN = 128;
constexpr int NT = 256;
constexpr int RBL = 2, CBL = 2;
constexpr int MAX_SLICES = 8;

struct Args {
  const uint16_t* A[2];
  int64_t width;          // columns of A in one segment (a multiple of 8)
  int chunks;             // chunks of 64 in one segment
  int segments;           // 1 or 2
  int M;
};

// 80 KB: A's chunks in a ring of three, the weights' in two
struct __attribute__((aligned(16))) ChunkA {
  uint4 v[BM * 8];
};
struct __attribute__((aligned(16))) ChunkB {
  uint4 v[BN * 8];
};

// slices of the reduction for a number of tiles
inline int slices(int64_t tiles, int64_t chunks) {
  return int(std::min<int64_t>({std::max<int64_t>(1, 512 / tiles), MAX_SLICES,
                                std::max<int64_t>(1, chunks / 4)}));
}

// The same with 16 to 32 slices, of at least eight chunks each, where the tiles leave
// room for them: 65 rows 8192 -> 512 14.1 us (with 8 slices 18.7), 128 rows 12288 -> 2048
// 22.0 (27.1).  Slices of four chunks: 65 rows 4096 -> 4096 21.6 us and with 8 slices 17.6,
// since their sums are 16 MB; 9 to 15 slices, which the second launch loads in two turns
// as well, gain nothing (10 of 333 rows 8192 -> 2064: 32.6 us, 8: 31.9).
inline int fine_slices(int64_t tiles, int64_t chunks) {
  const int64_t S = std::min<int64_t>({512 / tiles, 32, chunks / 8});
  return S < 16 ? slices(tiles, chunks) : int(S);
}

// Two halves of four waves each, whose accumulators hold the sums over two parts of the
// reduction, add them up: half 0 keeps rows 0..31 of each wave's 64 and half 1 the others,
// in acc[0].  Each hands the rest on through its `b0` and `b1`.
__device__ __forceinline__ void add_halves(v16f (&acc)[RBL][CBL], int half, int wave, int lane,
                                           ChunkB (&b0)[2], ChunkB (&b1)[2], v16f (&out)[1][CBL]) {
  // 8 KB a wave, two waves to an object
  auto at = [&](int h, int k) __attribute__((always_inline)) -> v4f* {
    return reinterpret_cast<v4f*>(wave < 2 ? b0[h].v : b1[h].v) + (wave & 1) * 512 + k * 64 + lane;
  };
#pragma unroll
  for (int j = 0; j < CBL; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v4f v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = half ? acc[0][j][4 * k + e] : acc[1][j][4 * k + e];
      *at(half, 4 * j + k) = v;
    }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < CBL; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const v4f v = *at(half ^ 1, 4 * j + k);
      // (half 0's sum first, in both halves)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[0][j][4 * k + e] = half ? v[e] + acc[1][j][4 * k + e] : acc[0][j][4 * k + e] + v[e];
    }
}

// Weights: fetch<set>(chunk) loads this thread's share of a chunk's B rows into
// one of two register sets, put<set, q>(b) dequantizes quarter q of it and (at
// the latest in quarter 3) writes it to LDS, slot(row, piece) is where piece
// `piece` of B row `row` lies.
using I0 = std::integral_constant<int, 0>;
using I1 = std::integral_constant<int, 1>;
using I2 = std::integral_constant<int, 2>;
using I3 = std::integral_constant<int, 3>;

template <class Weights>
__device__ __forceinline__ void tile_product(const Args& p, int64_t m0, int c0, int c1, Weights& w,
                                             ChunkA& a0, ChunkA& a1, ChunkA& a2, ChunkB& b0,
                                             ChunkB& b1, v16f (&acc)[RBL][CBL],
                                             int tid = int(threadIdx.x)) {
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int h = lane >> 5, r32 = lane & 31;
  // wave w brings rows 32 w .. 32 w + 31 of A, 8 rows to a transfer; rows past
  // the edge repeat the last row, pieces past the width the last piece
  // (addresses as in the wide tile: a uniform base and 32-bit offsets in bytes)
  uint32_t aoff[4], apiece[2];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = 32 * wave + 8 * t + (lane >> 3);
    aoff[t] = 2 * uint32_t(min(int64_t(r), p.M - 1 - m0)) * uint32_t(p.width);
    if (t < 2) apiece[t] = 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  const uint8_t* const base0 = reinterpret_cast<const uint8_t*>(p.A[0] + m0 * p.width);
  const uint8_t* const base1 = reinterpret_cast<const uint8_t*>(p.A[1] + m0 * p.width);
  auto dma = [&](int c, ChunkA& st) __attribute__((always_inline)) {
    c = min(c, c1 - 1);
    const bool second = c >= p.chunks;
    const int col = min(64 * (second ? c - p.chunks : c), int(p.width) - 8);
    const uint32_t last = 2 * uint32_t(int(p.width) - 8 - col);
    const uint8_t* const A = (second ? base1 : base0) + 2 * col;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      __builtin_amdgcn_global_load_lds(A + (aoff[t] + min(apiece[t & 1], last)),
                                       (lds_ptr_t)&st.v[(32 * wave + 8 * t) * 8], 16, 0, 0);
  };
  const int sw = (r32 >> 1) & 7;
  const int abase = (wm * 64 + r32) * 8;
  // One chunk: every wave waits for its transfers of it (the four of the next
  // chunk may stay in flight, nothing is issued after them) and for its LDS
  // writes; past the barrier the chunk is complete and the buffers of the one
  // before are free.  The loads two chunks ahead go out, then the MFMAs with
  // the LDS reads, the next chunk's dequantization and its LDS writes between
  // them.  Past the last chunk the loads repeat it.
  auto step = [&](int c, auto SET, const ChunkA& ac, ChunkA& an, const ChunkB& bc, ChunkB& bn)
      __attribute__((always_inline)) {
    constexpr int set = decltype(SET)::value;
    __builtin_amdgcn_s_waitcnt(0x0070 | 4);     // vmcnt(4) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    w.template fetch<set>(min(c + 2, c1 - 1));
    __builtin_amdgcn_sched_barrier(0);          // the four transfers stay last
    dma(c + 2, an);
    __builtin_amdgcn_sched_barrier(0);
    v8bf fa[2][RBL], fb[2][CBL];
    auto frag = [&](int ks, int n) __attribute__((always_inline)) {
      if (n < 2)
        fb[ks & 1][n] =
            __builtin_bit_cast(v8bf, bc.v[Weights::slot(wn * 64 + 32 * n + r32, 2 * ks + h)]);
      else
        fa[ks & 1][n - 2] =
            __builtin_bit_cast(v8bf, ac.v[abase + 256 * (n - 2) + ((2 * ks + h) ^ sw)]);
    };
#pragma unroll
    for (int n = 0; n < 4; ++n) frag(0, n);
    auto quarter = [&](auto KS) __attribute__((always_inline)) {
      constexpr int ks = decltype(KS)::value;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int i = n / CBL, j = n % CBL;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[ks & 1][i], fb[ks & 1][j], acc[i][j],
                                                            0, 0, 0);
        if (ks < 3) frag(ks + 1, n);
        if (n == 1) w.template put<(set ^ 1), ks>(bn.v);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    quarter(I0{});
    quarter(I1{});
    quarter(I2{});
    quarter(I3{});
  };
  w.template fetch<0>(c0);
  w.template fetch<1>(min(c0 + 1, c1 - 1));
  __builtin_amdgcn_sched_barrier(0);
  dma(c0, a0);
  dma(c0 + 1, a1);
  w.template put<0, 0>(b0.v);
  w.template put<0, 1>(b0.v);
  w.template put<0, 2>(b0.v);
  w.template put<0, 3>(b0.v);
  int c = c0;
  for (; c + 6 <= c1; c += 6) {
    step(c, I0{}, a0, a2, b0, b1);
    step(c + 1, I1{}, a1, a0, b1, b0);
    step(c + 2, I0{}, a2, a1, b0, b1);
    step(c + 3, I1{}, a0, a2, b1, b0);
    step(c + 4, I0{}, a1, a0, b0, b1);
    step(c + 5, I1{}, a2, a1, b1, b0);
  }
  if (c < c1) step(c, I0{}, a0, a2, b0, b1);
  if (c + 1 < c1) step(c + 1, I1{}, a1, a0, b1, b0);
  if (c + 2 < c1) step(c + 2, I0{}, a2, a1, b0, b1);
  if (c + 3 < c1) step(c + 3, I1{}, a0, a2, b1, b0);
  if (c + 4 < c1) step(c + 4, I0{}, a1, a0, b0, b1);
  // the repeated last transfers, before the buffers are used for anything else
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
}

}  // namespace svdq_mid

// Which of the forms takes which rows of a call with more than 64: the first
// `wide` rows the 256 x 256 tiles on weights dequantized up front, the others
// (up to 64 of them) the few-row form or the 128 x 128 tiles.  The wide form has
// the higher rate, but pays the dequantization and whole rounds of 256 tiles (one
// to a compute unit): 4099 rows to 12288 columns over 4096 are 816 tiles, four
// rounds and 422 us, or 4096 rows in three rounds and 3 rows apart, 372 us; 1000
// rows of the gated pair 4096 -> 12288 take 237 us in 128 x 128 tiles and 268 us in
// 256 x 256.  The times below are what the forms measured, in us: a round of 256
// wide tiles 1.72 a chunk of 64, a round of 512 tiles of 128 x 128 1.25, the
// dequantization 5.2 TB/s, sums of slices 4.5 TB/s, few rows their weights at
// 4.5 TB/s; 3 for a launch.
// few_us is the time of a few rows; 64 take about twice that (gated pair 4096 -> 12288:
// 18.6 here, 15 measured at one row, 28 at 33 and 35 at 64; linear gradient 12288 x
// 4096: 12.3, 14, 26 and 35).  A factor 1 + rows / 43, which fits them, changes the
// choice for 0.2% of sizes; on 24 of those it was 0.83 to 1.26 times as fast, 0.998 in
// the geometric mean (gated 0.96, its backward 0.95, linear gradient 1.06), since the
// estimates of the other forms are off by as much there.  It is left out.
namespace svdq_plan {

struct Shape {
  int64_t chunks;         // of the reduction
  int64_t wide_n, mid_n;  // tiles across
  int64_t weights;        // 4-bit weights of the call
  bool twin = false;      // whether a medium number of rows has the choice of medium()
};

inline double few_us(const Shape& p) { return 6 + 0.5625 * double(p.weights) / 4.5e6; }

inline double mid_us(int64_t rows, const Shape& p) {
  const int64_t tiles = (rows + 127) / 128 * p.mid_n;
  const int S = svdq_mid::slices(tiles, p.chunks);
  const double t = 3 + 1.25 * double((tiles * S + 511) / 512) * double(p.chunks) / S;
  return S == 1 ? t : t + 3 + 8.0 * S * double(rows) * double(p.mid_n) * 128 / 4.5e6;
}

// A medium number of rows where a tile may also go to two sets of four waves, each with
// half of a slice's chunks, which meet in LDS: as many waves, and half the partial sums
// or none.  500 rows 1024 -> 8192 take 19.0 us so and 29.8 in twice as many workgroups of one
// set, 333 rows 2048 -> 8192 27.3 and 31.7, 900 rows 4096 -> 4096 48.3 and 54.2; but 333 rows
// 4096 -> 4096, whose 96 tiles in two slices fill three quarters of the chip, 29.9 and
// 28.3, and more tiles than compute units leave the last round emptier: 400 rows 2048 ->
// 16384 53.7 and 48.9.  The constants are fitted to such pairs: a chunk 1.25 us with two
// sets on a compute unit, 0.9 with one, two chunks of a twin 1.35, the sums of slices 6 TB/s.
struct Medium {
  int S;
  bool twin;
  double us;
};

inline Medium medium(int64_t rows, const Shape& p) {
  const int64_t tiles = (rows + 127) / 128 * p.mid_n;
  const double sums = 8.0 * double(rows) * double(p.mid_n) * 128 / 6e6, c = double(p.chunks);
  const int S = svdq_mid::fine_slices(tiles, p.chunks);
  Medium m{S, false, (S == 1 ? 3 : 6 + S * sums) +
                         (tiles * S <= 256 ? 0.9 : 1.25) * double((tiles * S + 511) / 512) * c / S};
  // (a slice has a chunk for each set)
  const int most = int(std::min<int64_t>({256 / tiles, 16, p.chunks / 2}));
  for (int s = 1; s <= most; ++s) {
    const double us = (s == 1 ? 5 : 8 + s * sums) + 0.675 * c / s;
    if (us < m.us) m = {s, true, us};
  }
  return m;
}

inline double wide_us(int64_t rows, const Shape& p) {
  const int64_t tiles = (rows + 255) / 256 * p.wide_n;
  return 6 + 1.72 * double((tiles + 255) / 256) * double(p.chunks) +
         2.5625 * double(p.weights) / 5.2e6;
}

inline double rest_us(int64_t rows, const Shape& p) {
  return rows == 0     ? 0
         : rows <= 64 ? few_us(p)
         : p.twin     ? medium(rows, p).us
                      : mid_us(rows, p);
}

// all rows in the wide form with the last round split (gemm_bf16.h's Rounds); its join
// writes and reads the sums
inline double split_us(const svdq_gemm::Rounds& r, const Shape& p) {
  return 9 + 1.72 * (double(r.full / svdq_gemm::UNITS) + 1.0 / r.S) * double(p.chunks) +
         2.5625 * double(p.weights) / 5.2e6 + double(svdq_gemm::rounds_bytes(r)) * 2 / 4.5e6;
}

// rows of the wide form: 0, all, or whole tiles that leave the last round out
inline int64_t wide_rows(int64_t M, const Shape& p, double* us = nullptr) {
  int64_t best = 0;
  double t = rest_us(M, p);
  auto consider = [&](int64_t m) {
    const double u = wide_us(m, p) + rest_us(M - m, p);
    if (u < t) t = u, best = m;
  };
  consider(M);
  const int64_t whole = M / 256 * 256;
  for (int64_t i = 0; i < 32 && whole - 256 * i > 0; ++i) consider(whole - 256 * i);
  if (us) *us = t;
  return best;
}

}  // namespace svdq_plan
