// Gated feed-forward pair of AWQ W4A16 layers (gfx950):
//
//   G = X Wg^T + bg,  U = X Wu^T + bu,  H = act(G) * U
//
// Wg, Wu [N, K] in the AWQ format (weights bf16((q - z) s)), X bf16 [M, K].
// G and U stay in the fp32 accumulators of the bf16 MFMAs; the activation and
// the product are computed there in fp32, and H is rounded once.  For a
// backward pass G and U can be stored too, rounded to bf16 (half the bytes,
// and what a pair of separate layers would hand on).

#include "gemm_bf16.h"

using namespace svdq_dev;

namespace {

// The G and U of R blocks of 32 rows and 32 columns in a wave's accumulators:
// bias, activation, product, and the stores through the wave's LDS buffer `eb`
// (32 x 36 floats).
template <int ACT, int R>
__device__ __forceinline__ void gated_epilogue(v16f (&acc)[R][2], float* eb, int lane, int64_t row0,
                                               int64_t col0, int M, int N,
                                               const uint16_t* __restrict__ bg,
                                               const uint16_t* __restrict__ bu, void* H, bool hbf16,
                                               uint16_t* Gs, uint16_t* Us) {
  const int64_t n = col0 + (lane & 31);
  const float vg = bg && n < N ? bf16_to_f32(bg[n]) : 0.f;
  const float vu = bu && n < N ? bf16_to_f32(bu[n]) : 0.f;
  const float none[1] = {0.f};
  v16f o[R][1];
  auto store = [&](void* Y, bool b16) {
    if (b16)
      store_wave_tile<R, 1, true>(o, none, eb, lane, row0, col0, M, N, Y);
    else
      store_wave_tile<R, 1, false>(o, none, eb, lane, row0, col0, M, N, Y);
  };
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      acc[i][0][e] += vg;
      acc[i][1][e] += vu;
    }
  if (Gs) {
#pragma unroll
    for (int i = 0; i < R; ++i) o[i][0] = acc[i][0];
    store(Gs, true);
#pragma unroll
    for (int i = 0; i < R; ++i) o[i][0] = acc[i][1];
    store(Us, true);
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][0][e] = gate_act<ACT>(acc[i][0][e]) * acc[i][1][e];
  store(H, hbf16);
}

// ----------------------------------------------------------- few rows
// Up to 64 rows the time is the weights' way from memory, and how many launches
// follow one another.  Small products take one launch (gated_column_kernel).
// Larger ones take two: a workgroup's 8 waves own 16 columns of both weights each,
// all rows, and one of S slices of K; X's slice is in LDS, the weights stream
// through registers D chunks ahead.  The slices' partial G and U [S][2][M][N] are
// joined by gated_sum_kernel, which applies bias, activation and product.

constexpr int ROWS = 64;                 // the most rows of this form
constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int D = 2;
constexpr int LDS_X = 64 << 10;
constexpr int SUM_SLICES = 8;            // slices that the second launch loads at once

// The two-launch form, 64 rows 4096 -> 12288: 34 us (X and the partial sums in the
// L2 and the dequantization share the time).
struct Split {
  int blocks, slices;
};

// About 512 workgroups, two to a compute unit.  Above 16 rows the partial sums
// are more than the weights, so there are at most 4 slices: 33 rows 2048 -> 5456
// took 14.2 us in 8 and 13.1 in 4 (one row 4096 -> 12288, 15.7 in 5 and 17.6 in 4);
// but narrow layers, where that leaves most of the chip idle, get more, of at least 4
// chunks, up to 128 workgroups.
Split split(int64_t M, int64_t K, int64_t N) {
  Split p;
  p.blocks = int((N + 16 * WAVES - 1) / (16 * WAVES));
  p.slices = int(std::min<int64_t>(
      {K / 64, M > 16 ? SUM_SLICES / 2 : SUM_SLICES, std::max<int64_t>(1, 512 / p.blocks)}));
  if (M > 16) p.slices = std::max(p.slices, int(std::min<int64_t>({K / 256, 32, 128 / p.blocks})));
  return p;
}

// Whether few rows take one launch (gated_column_kernel), where every 16 columns
// read all of X: N / 16 times 2 M K bytes from the L2.  Measured: 20 rows
// 4096 -> 12288 (M N K = 1.0e9) 22 us either way, one row 13.8 against 16.2, 20
// rows 1024 -> 2048 4.0 against 7.9, but 64 rows 4096 -> 12288 49 against 34.  On
// more than 16 rows a long K and few columns take too long in the N / 16 workgroups:
// 33 rows 8192 -> 512 20.9 against 12.3, 64 rows 4096 -> 1024 17.9 against 13.1 (20
// rows 4096 -> 512 8.6 against 8.8, and 33 rows 4096 -> 2048 stay at 12.1).
bool one_launch(int64_t M, int64_t K, int64_t N) {
  return M * N <= (int64_t(1) << 30) / K && !(M > 16 && K >= 4096 && N <= 1024);
}

template <int MT>
__global__ __launch_bounds__(NT, 4) void gated_slice_kernel(
    const uint16_t* __restrict__ X, int M, int K, int N, svdq::AwqWeight wg, svdq::AwqWeight wu,
    int S, int sub, float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int G = K / 64;
  const int slice = blockIdx.x % S;
  const int g0 = int(int64_t(slice) * G / S), count = int(int64_t(slice + 1) * G / S) - g0;
  const int64_t n = (int64_t(blockIdx.x / S) * WAVES + wave) * 16 + r;
  const int64_t nc = min(n, int64_t(N) - 1);

  // lane group j holds the codes k = 16 j .. 16 j + 15 of its row's chunk
  struct Slot {
    uint2 w[2];
    uint32_t s[2], z[2];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's
  // data), so that the number of loads in flight is fixed
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int64_t at = int64_t(g0 + min(i, count - 1)) * N + nc;
    sl.w[0] = *reinterpret_cast<const uint2*>(wg.q + at * 32 + 8 * j);
    sl.w[1] = *reinterpret_cast<const uint2*>(wu.q + at * 32 + 8 * j);
    sl.s[0] = wg.s[at];
    sl.z[0] = wg.z[at];
    sl.s[1] = wu.s[at];
    sl.z[1] = wu.z[at];
  };
  v4f acc[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[mt][t] = v4f{0, 0, 0, 0};

  // `sub` chunks of X at a time in LDS: rows of `sub` chunks and 16 bytes, so
  // that 16 rows start in 16 different groups of 4 banks
  const int rowb = sub * 128 + 16;
  int xoff[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xoff[mt] = min(16 * mt + r, M - 1) * rowb + 32 * j;
  for (int c0 = 0; c0 < count; c0 += sub) {
    const int here = min(sub, count - c0);
    if (c0) __syncthreads();
    for (int i = tid; i < M * here * 8; i += NT) {
      const int m = i / (here * 8), o = i - m * (here * 8);
      *reinterpret_cast<uint4*>(lds + m * rowb + 16 * o) =
          *reinterpret_cast<const uint4*>(X + int64_t(m) * K + 64 * int64_t(g0 + c0) + 8 * o);
    }
    if (c0 == 0)
#pragma unroll
      for (int d = 0; d < D; ++d) fetch(d, ring[d]);
    // (not __syncthreads, which would wait for the weights too)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    for (int c = 0; c < here; c += D)
#pragma unroll
      for (int d = 0; d < D; ++d) {
        Slot& sl = ring[d];
        // past the last chunk the scales are zeros
        const bool live = c + d < here;
        v8bf b[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float s = live ? __uint_as_float(sl.s[t] << 16) : 0.f;
          const float zs = -__uint_as_float(sl.z[t] << 16) * s;
          b[t][0] = __builtin_bit_cast(v8bf, dequant8(sl.w[t].x, s, zs));
          b[t][1] = __builtin_bit_cast(v8bf, dequant8(sl.w[t].y, s, zs));
        }
        const uint8_t* const xc = lds + 128 * min(c + d, here - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v8bf a = *reinterpret_cast<const v8bf*>(xc + xoff[mt] + 16 * h);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[t][h], acc[mt][t], 0, 0, 0);
          }
        fetch(c0 + c + d + D, sl);
      }
  }
  if (n >= N) return;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = 16 * mt + 4 * j + e;
        // (read by the next launch, on any XCD: past this one's L2 at once)
        if (m < M)
          __builtin_nontemporal_store(acc[mt][t][e],
                                      part + ((int64_t(slice) * 2 + t) * M + m) * N + n);
      }
}

// One launch: a workgroup owns 16 columns of both weights, its 8
// waves take the chunks of K in turn, each with its own piece of X, and the
// sums meet in LDS.  Bound by the weights' way from memory: one row
// 4096 -> 12288 (56.6 MB) 13.7 us, 4.1 TB/s; 33 rows 2048 -> 5456 12.8 us; one row
// 1024 -> 2048 3.0 us, most of it the launch.
template <int MT, int ACT>
__global__ __launch_bounds__(NT, MT == 1 ? 6 : 4) void gated_column_kernel(
    const uint16_t* __restrict__ X, int M, int K, int N, svdq::AwqWeight wg, svdq::AwqWeight wu,
    const uint16_t* __restrict__ bg, const uint16_t* __restrict__ bu, void* __restrict__ H,
    bool hbf16, uint16_t* __restrict__ Gs, uint16_t* __restrict__ Us) {
  __shared__ v4f red[WAVES][2 * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int64_t n = int64_t(blockIdx.x) * 16 + r;                   // (N is a multiple of 16)
  const int G = K / 64, count = (G - wave + WAVES - 1) / WAVES;     // chunks of this wave
  const uint16_t* xrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xrow[mt] = X + int64_t(min(16 * mt + r, M - 1)) * K + 16 * j;
  struct Slot {
    uint2 w[2];
    uint32_t s[2], z[2];
    uint4 x[MT][2];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's
  // data; a wave without chunks loads chunk 0 and never uses it)
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int c = count > 0 ? wave + WAVES * min(i, count - 1) : 0;
    const int64_t at = int64_t(c) * N + n;
    sl.w[0] = *reinterpret_cast<const uint2*>(wg.q + at * 32 + 8 * j);
    sl.w[1] = *reinterpret_cast<const uint2*>(wu.q + at * 32 + 8 * j);
    sl.s[0] = wg.s[at];
    sl.z[0] = wg.z[at];
    sl.s[1] = wu.s[at];
    sl.z[1] = wu.z[at];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4* const x = reinterpret_cast<const uint4*>(xrow[mt] + 64 * int64_t(c));
      sl.x[mt][0] = x[0];
      sl.x[mt][1] = x[1];
    }
  };
  v4f acc[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[mt][t] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, ring[d]);
  for (int c = 0; c < count; c += D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Slot& sl = ring[d];
      // past the last chunk the scales are zeros (which leaves an infinite X a NaN;
      // zeros for X too cost 33 rows 2048 -> 5456 0.7 us)
      const bool live = c + d < count;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float s = live ? __uint_as_float(sl.s[t] << 16) : 0.f;
        const float zs = -__uint_as_float(sl.z[t] << 16) * s;
        const v8bf b0 = __builtin_bit_cast(v8bf, dequant8(sl.w[t].x, s, zs));
        const v8bf b1 = __builtin_bit_cast(v8bf, dequant8(sl.w[t].y, s, zs));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, sl.x[mt][0]), b0, acc[mt][t], 0, 0, 0);
          acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, sl.x[mt][1]), b1, acc[mt][t], 0, 0, 0);
        }
      }
      fetch(c + d + D, sl);
    }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < 2; ++t) red[wave][2 * mt + t][lane] = acc[mt][t];
  __syncthreads();
  if (wave >= MT) return;
  v4f v[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    v[t] = red[0][2 * wave + t][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v[t] += red[w][2 * wave + t][lane];
    const uint16_t* const b = t ? bu : bg;
    if (b) v[t] += bf16_to_f32(b[n]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t m = 16 * wave + 4 * j + e;
    if (m >= M) continue;
    const float h = gate_act<ACT>(v[0][e]) * v[1][e];
    if (hbf16)
      static_cast<uint16_t*>(H)[m * N + n] = f32_to_bf16(h);
    else
      static_cast<float*>(H)[m * N + n] = h;
    if (Gs) {
      Gs[m * N + n] = f32_to_bf16(v[0][e]);
      Us[m * N + n] = f32_to_bf16(v[1][e]);
    }
  }
}

// 4 columns per thread
template <int ACT>
__global__ __launch_bounds__(64) void gated_sum_kernel(
    const float* __restrict__ part, int S, int M, int N, const uint16_t* __restrict__ bg,
    const uint16_t* __restrict__ bu, void* __restrict__ H, bool hbf16, uint16_t* __restrict__ Gs,
    uint16_t* __restrict__ Us) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x, total = int64_t(M) * N / 4;
  if (i >= total) return;
  const int64_t n = 4 * i % N;
  // all loads first; a slice past the last counts as zeros
  v4f v[SUM_SLICES][2];
#pragma unroll
  for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      v[q][t] = reinterpret_cast<const v4f*>(part)[(2 * int64_t(min(q, S - 1)) + t) * total + i];
  // (a bias is aligned to its elements only: a copy leaves the compiler to choose loads
  // that the target takes at any address)
  uint16_t b[2][4] = {};
  if (bg) __builtin_memcpy(b[0], bg + n, 8);
  if (bu) __builtin_memcpy(b[1], bu + n, 8);
  __builtin_amdgcn_sched_barrier(0);
  v4f p[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    p[t] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[t][e] += q < S ? v[q][t][e] : 0.f;
  }
  for (int q0 = SUM_SLICES; q0 < S; q0 += SUM_SLICES) {
#pragma unroll
    for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        v[q][t] =
            reinterpret_cast<const v4f*>(part)[(2 * int64_t(min(q0 + q, S - 1)) + t) * total + i];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[t][e] += q0 + q < S ? v[q][t][e] : 0.f;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) p[t][e] += bf16_to_f32(b[t][e]);
  v4f h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = gate_act<ACT>(p[0][e]) * p[1][e];
  auto pack = [](v4f x) { return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); };
  if (hbf16)
    static_cast<uint2*>(H)[i] = pack(h);
  else
    static_cast<v4f*>(H)[i] = h;
  if (Gs) {
    reinterpret_cast<uint2*>(Gs)[i] = pack(p[0]);
    reinterpret_cast<uint2*>(Us)[i] = pack(p[1]);
  }
}

// ---------------------------------------------------------- many rows
// The weights are dequantized once into the workspace, 32 rows of Wg and the
// 32 rows of Wu with the same n alternating, so that one wave's two column
// blocks of the product are the G and the U of the same outputs.

// 64 rows of the pair matrix and four groups of 64 k (two stages each) per
// workgroup (2 x 12288 x 4096: 258 MB in 49 us, 5.3 TB/s; one group per workgroup,
// with fewer loads in flight, took 62); rows past N are zeros.  Four lanes take
// one row, 8 k of each stage, so that a wave stores 1 KB in a row.
constexpr int DEQUANT_GROUPS = 4;

__global__ __launch_bounds__(256) void pair_dequant_kernel(svdq::AwqWeight wg, svdq::AwqWeight wu,
                                                           int K, int N,
                                                           uint16_t* __restrict__ B) {
  const int row = threadIdx.x >> 2, piece = threadIdx.x & 3;
  const int blocks = (N + 31) / 32, G = K / 64, g0 = blockIdx.x / blocks * DEQUANT_GROUPS;
  const int64_t block = blockIdx.x % blocks, n = block * 32 + (row & 31);
  const svdq::AwqWeight w = row >= 32 ? wu : wg;
  // (rows past N read the last row and groups past K the last group)
  const int64_t nc = min(n, int64_t(N) - 1);
  uint32_t c[DEQUANT_GROUPS][2];
  uint16_t s[DEQUANT_GROUPS], z[DEQUANT_GROUPS];
#pragma unroll
  for (int i = 0; i < DEQUANT_GROUPS; ++i) {
    const int64_t at = int64_t(min(g0 + i, G - 1)) * N + nc;
    const uint32_t* const p = reinterpret_cast<const uint32_t*>(w.q + at * 32 + piece * 4);
    c[i][0] = p[0];
    c[i][1] = p[4];
    s[i] = w.s[at];
    z[i] = w.z[at];
  }
#pragma unroll
  for (int i = 0; i < DEQUANT_GROUPS; ++i) {
    if (g0 + i >= G) break;
    const float f = n < N ? bf16_to_f32(s[i]) : 0.f, fz = -bf16_to_f32(z[i]) * f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      *svdq_gemm::weight_at(B, K / 32, block * 64 + row, 64 * (g0 + i) + 32 * t + 8 * piece) =
          dequant8(c[i][t], f, fz);
  }
}

template <int ACT>
__global__ __launch_bounds__(svdq_gemm::NT) void gated_wide_kernel(
    svdq_gemm::Args p, int N, const uint16_t* __restrict__ bg, const uint16_t* __restrict__ bu,
    void* __restrict__ H, bool hbf16, uint16_t* __restrict__ Gs, uint16_t* __restrict__ Us) {
  using namespace svdq_gemm;
  __shared__ Stage st0, st1, st2, st3, st4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  int64_t m0, b0;
  tile_origin((p.M + BM - 1) / BM, (p.rows + BN - 1) / BN, BM, BN, m0, b0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  tile_product(p, m0, b0, st0, st1, st2, st3, st4, acc);

  gated_epilogue<ACT>(acc, epilogue_buffer<32 * 36>(wave, st0, st1, st2), lane, m0 + wm * WM,
                      b0 / 2 + wn * 32, p.M, N, bg, bu, H, hbf16, Gs, Us);
}

// -------------------------------------------------------- medium number of rows
// B rows of a tile: for each of the two wave columns 32 rows of Wg and the 32
// rows of Wu with the same n.  Two threads take one row, 32 codes each.
struct PairWeights {
  svdq::AwqWeight wg, wu;
  // this thread's row of chunk 0; a chunk further is N rows further
  const uint8_t* q;
  const uint16_t *s, *z;
  int N, row, half;
  uint4 c[2];
  uint16_t cs[2], cz[2];

  __device__ __forceinline__ PairWeights(const svdq::AwqWeight& g, const svdq::AwqWeight& u, int N,
                                         int64_t n0)
      : N(N), row(int(threadIdx.x) >> 1), half(threadIdx.x & 1) {
    const bool up = row & 32;
    const int64_t nr = min(n0 + (row >> 6) * 32 + (row & 31), int64_t(N) - 1);
    q = (up ? u.q : g.q) + nr * 32 + 16 * half;
    s = (up ? u.s : g.s) + nr;
    z = (up ? u.z : g.z) + nr;
  }
  static __device__ __forceinline__ int slot(int row, int piece) {
    return row * 8 + (piece ^ ((row >> 1) & 7));
  }
  template <int set>
  __device__ __forceinline__ void fetch(int chunk) {
    const int64_t at = int64_t(chunk) * N;
    c[set] = *reinterpret_cast<const uint4*>(q + at * 32);
    cs[set] = s[at];
    cz[set] = z[at];
  }
  template <int set, int i>
  __device__ __forceinline__ void put(uint4* b) {
    const uint32_t w = i == 0 ? c[set].x : i == 1 ? c[set].y : i == 2 ? c[set].z : c[set].w;
    const float f = bf16_to_f32(cs[set]);
    b[slot(row, 4 * half + i)] = dequant8(w, f, -bf16_to_f32(cz[set]) * f);
  }
};

template <int ACT>
__global__ __launch_bounds__(svdq_mid::NT, 2) void gated_mid_kernel(
    svdq_mid::Args p, svdq::AwqWeight wg, svdq::AwqWeight wu, int N, int S, int tiles,
    const uint16_t* __restrict__ bg, const uint16_t* __restrict__ bu, void* __restrict__ H,
    bool hbf16, uint16_t* __restrict__ Gs, uint16_t* __restrict__ Us, float* __restrict__ part) {
  using namespace svdq_mid;
  __shared__ ChunkA a0, a1, a2;
  __shared__ ChunkB b0, b1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = blockIdx.x / tiles;
  int64_t m0, n0;
  tile_at(int(blockIdx.x % tiles), (p.M + BM - 1) / BM, (N + 63) / 64, BM, 64, m0, n0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  PairWeights w(wg, wu, N, n0);
  tile_product(p, m0, int(int64_t(slice) * p.chunks / S), int(int64_t(slice + 1) * p.chunks / S), w,
               a0, a1, a2, b0, b1, acc);
  const int64_t row0 = m0 + (wave >> 1) * 64, col0 = n0 + (wave & 1) * 32;
  float* const eb = reinterpret_cast<float*>(wave < 3 ? &a0 : &a1) + (wave % 3) * (32 * 36);
  if (S == 1) {
    gated_epilogue<ACT>(acc, eb, lane, row0, col0, p.M, N, bg, bu, H, hbf16, Gs, Us);
    return;
  }
  const float none[1] = {0.f};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    v16f o[RBL][1];
#pragma unroll
    for (int i = 0; i < RBL; ++i) o[i][0] = acc[i][t];
    store_wave_tile<RBL, 1, false>(o, none, eb, lane, row0, col0, p.M, N,
                                   part + (int64_t(slice) * 2 + t) * p.M * N);
  }
}

int64_t pair_rows(int64_t N) { return (N + 31) / 32 * 64; }
int64_t mid_tiles(int64_t M, int64_t N) { return (M + 127) / 128 * ((N + 63) / 64); }

int64_t wide_rows(int64_t M, int64_t K, int64_t N) {
  if (M <= ROWS) return 0;
  return svdq_plan::wide_rows(M, {K / 64, (pair_rows(N) + 255) / 256, (N + 63) / 64, 2 * K * N});
}

size_t pair_bytes(int64_t K, int64_t N) {
  return svdq_gemm::weight_bytes(pair_rows(N), K / 32);
}

// bytes of the partial sums of `rows` rows
size_t part_bytes(int64_t rows, int64_t K, int64_t N) {
  if (rows == 0 || (rows <= ROWS && one_launch(rows, K, N))) return 0;
  const int S = rows <= ROWS ? split(rows, K, N).slices
                             : svdq_mid::slices(mid_tiles(rows, N), K / 64);
  return rows > ROWS && S == 1 ? 0 : svdq::align256(size_t(S) * 2 * size_t(rows) * size_t(N) * 4);
}

// A call's rows [m0, m0 + M)
struct Call {
  const uint16_t* X;
  int64_t M, K, N;
  svdq::AwqWeight wg, wu;
  const uint16_t *bg, *bu;
  bool silu;
  void* H;
  bool hbf16;
  uint16_t *G, *U;
  hipStream_t s;

  Call rows(int64_t m0, int64_t m) const {
    Call c = *this;
    c.X += m0 * K;
    c.M = m;
    c.H = static_cast<uint8_t*>(H) + m0 * N * (hbf16 ? 2 : 4);
    if (G) {
      c.G += m0 * N;
      c.U += m0 * N;
    }
    return c;
  }
};

svdq_status sum(const Call& c, const float* part, int S) {
  auto k = c.silu ? gated_sum_kernel<SVDQ_SILU> : gated_sum_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(unsigned((c.M * c.N / 4 + 63) / 64)), dim3(64), 0, c.s, part, S,
                     int(c.M), int(c.N), c.bg, c.bu, c.H, c.hbf16, c.G, c.U);
  return svdq::check_launch("gated_sum");
}

template <int MT>
svdq_status slices(const Call& c, float* part) {
  const Split p = split(c.M, c.K, c.N);
  // chunks of X that fit LDS (64 rows: 6 chunks of 128 bytes).  A multiple of D: chunk
  // c of a piece is in slot c % D of the register ring, which goes on over the pieces.
  const int most = int((LDS_X / c.M - 16) / 128 / D * D);
  const int len = int((c.K / 64 + p.slices - 1) / p.slices);
  const int sub = std::min(most, (len + D - 1) / D * D);
  hipLaunchKernelGGL(gated_slice_kernel<MT>, dim3(unsigned(p.blocks * p.slices)), dim3(NT),
                     size_t(c.M) * (sub * 128 + 16), c.s, c.X, int(c.M), int(c.K), int(c.N), c.wg,
                     c.wu, p.slices, sub, part);
  return svdq::check_launch("gated_slice");
}

template <int MT>
svdq_status columns(const Call& c) {
  auto k = c.silu ? gated_column_kernel<MT, SVDQ_SILU> : gated_column_kernel<MT, SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(unsigned(c.N / 16)), dim3(NT), 0, c.s, c.X, int(c.M), int(c.K),
                     int(c.N), c.wg, c.wu, c.bg, c.bu, c.H, c.hbf16, c.G, c.U);
  return svdq::check_launch("gated_column");
}

svdq_status few(const Call& c, float* part) {
  if (one_launch(c.M, c.K, c.N)) switch ((c.M + 15) / 16) {
      case 1: return columns<1>(c);
      case 2: return columns<2>(c);
      case 3: return columns<3>(c);
      default: return columns<4>(c);
    }
  switch ((c.M + 15) / 16) {
    case 1: SVDQ_TRY(slices<1>(c, part)); break;
    case 2: SVDQ_TRY(slices<2>(c, part)); break;
    case 3: SVDQ_TRY(slices<3>(c, part)); break;
    default: SVDQ_TRY(slices<4>(c, part)); break;
  }
  return sum(c, part, split(c.M, c.K, c.N).slices);
}

svdq_status mid(const Call& c, float* part) {
  const int64_t tiles = mid_tiles(c.M, c.N);
  const int S = svdq_mid::slices(tiles, c.K / 64);
  svdq_mid::Args p{{c.X, c.X}, c.K, int(c.K / 64), 1, int(c.M)};
  auto k = c.silu ? gated_mid_kernel<SVDQ_SILU> : gated_mid_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(unsigned(tiles * S)), dim3(svdq_mid::NT), 0, c.s, p, c.wg, c.wu,
                     int(c.N), S, int(tiles), c.bg, c.bu, c.H, c.hbf16, c.G, c.U, part);
  SVDQ_TRY(svdq::check_launch("gated_mid"));
  return S == 1 ? SVDQ_OK : sum(c, part, S);
}

svdq_status wide(const Call& c, uint16_t* B) {
  const int64_t quads = (c.K / 64 + DEQUANT_GROUPS - 1) / DEQUANT_GROUPS;
  hipLaunchKernelGGL(pair_dequant_kernel, dim3(unsigned((c.N + 31) / 32 * quads)), dim3(256), 0,
                     c.s, c.wg, c.wu, int(c.K), int(c.N), B);
  SVDQ_TRY(svdq::check_launch("pair_dequant"));
  const int64_t rows = pair_rows(c.N), tiles = (c.M + 255) / 256 * ((rows + 255) / 256);
  svdq_gemm::Args p{{c.X, c.X}, c.K, int(c.K / 64), 1, B, int(c.M), int(rows)};
  auto k = c.silu ? gated_wide_kernel<SVDQ_SILU> : gated_wide_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(unsigned(tiles)), dim3(svdq_gemm::NT), 0, c.s, p, int(c.N), c.bg, c.bu,
                     c.H, c.hbf16, c.G, c.U);
  return svdq::check_launch("gated_wide");
}

}  // namespace

namespace svdq {

size_t awq_gated_workspace(int64_t M, int64_t K, int64_t N) {
  const int64_t w = wide_rows(M, K, N);
  return (w ? pair_bytes(K, N) : 0) + part_bytes(M - w, K, N);
}

svdq_status launch_awq_gated(const uint16_t* X, int64_t M, int64_t K, int64_t N, AwqWeight wg,
                             AwqWeight wu, const uint16_t* bg, const uint16_t* bu, svdq_act act,
                             void* H, svdq_dtype h_dt, uint16_t* G, uint16_t* U, void* ws,
                             hipStream_t s) {
  const Call c{X, M, K, N, wg, wu, bg, bu, act == SVDQ_SILU, H, h_dt == SVDQ_BF16, G, U, s};
  const int64_t w = wide_rows(M, K, N), rest = M - w;
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  if (w) SVDQ_TRY(wide(c.rows(0, w), reinterpret_cast<uint16_t*>(w8)));
  if (!rest) return SVDQ_OK;
  float* const part = reinterpret_cast<float*>(w8 + (w ? pair_bytes(K, N) : 0));
  return rest <= ROWS ? few(c.rows(w, rest), part) : mid(c.rows(w, rest), part);
}

}  // namespace svdq
