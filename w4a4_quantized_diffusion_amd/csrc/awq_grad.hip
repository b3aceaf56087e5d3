// Input gradients through frozen AWQ W4A16 weights (gfx950).
//
//   one layer    dX = dY wd
//   gated pair   dU = dH act(G),  dG = dH U act'(G),  dX = dG Wg + dU Wu
//
// wd = bf16((q - z) s) [N, K]; the reduction runs over the N outputs, across
// the rows of the 4-bit storage.  A thread that dequantizes the same k of
// eight consecutive rows n packs them over n, so the transposition costs
// nothing beyond the conversion to bf16, and the products run on bf16 MFMAs
// with fp32 sums.  dG and dU enter the products rounded to bf16 (the type
// they are returned in).

#include "gemm_bf16.h"

using namespace svdq_dev;

namespace {

// dG, dU of 8 elements per thread: memory-bound, 503 MB in 76 us (6.6 TB/s, part of
// it from the Infinity Cache) for 4096 x 12288
template <int ACT>
__global__ __launch_bounds__(256) void gate_grad_kernel(const uint16_t* __restrict__ dH,
                                                        const uint16_t* __restrict__ G,
                                                        const uint16_t* __restrict__ U,
                                                        int64_t n8, uint16_t* __restrict__ dG,
                                                        uint16_t* __restrict__ dU) {
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n8; i += step) {
    const uint4 h = reinterpret_cast<const uint4*>(dH)[i], g = reinterpret_cast<const uint4*>(G)[i],
                u = reinterpret_cast<const uint4*>(U)[i];
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w},
                   uw[4] = {u.x, u.y, u.z, u.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a0, d0, a1, d1;
      gate_act_grad<ACT>(__uint_as_float(gw[j] << 16), a0, d0);
      gate_act_grad<ACT>(__uint_as_float(gw[j] & 0xFFFF0000u), a1, d1);
      const float h0 = __uint_as_float(hw[j] << 16), h1 = __uint_as_float(hw[j] & 0xFFFF0000u);
      const float u0 = __uint_as_float(uw[j] << 16), u1 = __uint_as_float(uw[j] & 0xFFFF0000u);
      og[j] = pack_bf16x2(h0 * u0 * d0, h1 * u1 * d1);
      ou[j] = pack_bf16x2(h0 * a0, h1 * a1);
    }
    reinterpret_cast<uint4*>(dG)[i] = make_uint4(og[0], og[1], og[2], og[3]);
    reinterpret_cast<uint4*>(dU)[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// 8 rows n (from row index at = g N + n, n a multiple of 8) and the 8 k of
// dword j of a group, packed over n: out[i] holds k = 8j + i
__device__ __forceinline__ void transpose_dequant8(const svdq::AwqWeight& w, int64_t at, int j,
                                                   uint4 (&out)[8]) {
  const uint4 s4 = *reinterpret_cast<const uint4*>(w.s + at);
  const uint4 z4 = *reinterpret_cast<const uint4*>(w.z + at);
  const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w}, zw[4] = {z4.x, z4.y, z4.z, z4.w};
  uint32_t o[8][4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float v[2][8];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t c = *reinterpret_cast<const uint32_t*>(w.q + (at + 2 * p + r) * 32 + 4 * j);
      const float s = __uint_as_float(r ? sw[p] & 0xFFFF0000u : sw[p] << 16);
      const float zs = -__uint_as_float(r ? zw[p] & 0xFFFF0000u : zw[p] << 16) * s;
      dequant8_f32(c, s, zs, v[r]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][p] = pack_bf16x2(v[0][i], v[1][i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
}

// ----------------------------------------------------------- few rows
// Up to 64 rows the time is the weights' way from memory.  A workgroup takes
// 128 columns of dX (two groups) and one of S slices of the reduction, counted
// in steps of 32 n (a gated pair's steps run over both layers); its 8 waves
// take the steps in turn and meet in LDS.  Lane (j, r) of a wave dequantizes
// 8 k of the 8 rows n = 8 j .. 8 j + 7: column t of the 16 x 16 product t is
// k = 64 (r / 8) + 8 (r % 8) + t, so a lane's 8 products are 8 consecutive k.
// The rows' own operand (dY, or dG and dU computed here from dH, G and U) is
// in LDS.  Partial sums [S][M][K] are joined by grad_sum_kernel.
//
// A wave's loads, its two or three steps of products and the workgroup's reduction
// follow one another and nothing hides them (the dequantization, 2.6 vector
// instructions a code, is less than 2 us of it), so every compute unit is needed: one
// row 4096 x 4096 takes 7.5 us in 512 workgroups (6.4 and a launch of 2.6 for the
// sums), and 17 in the 32 that need no second launch.  Twenty rows of the pair 2048 x
// 5456 take 14 us.

constexpr int ROWS = 64;                 // the most rows of this form
constexpr int LDS_A = 64 << 10;          // for the rows' operand of 16 rows, twice that above
constexpr int MAX_SLICES = 16;
// Steps up to which the 16 waves of one workgroup take them all, and there is one
// launch: 512 outputs to 1024 columns 5.1 us against 5.9 in two launches, 1024
// outputs 6.9 against 6.0, where the host's 3 us for the second launch decide.
constexpr int ONE_SLICE = 32;

// The dG and dU of a gated pair's few rows are formed by every workgroup for its
// slice of n, so (K / 128) M N times 2; above this many (times 2) a launch of
// their own costs less: 40 rows 4096 x 8192 30.5 us against 39, 20 rows 2048 x
// 5456 14.7 against 14.0.
constexpr int64_t FUSED_GRADS = 4 << 20;

struct Split {
  int blocks, slices, waves;
};

Split split(int64_t M, int64_t K, int64_t N, int layers) {
  Split p;
  p.blocks = int((K + 127) / 128);
  const int64_t steps = (N + 31) / 32 * layers;
  p.waves = 8;
  if (M <= 16 && steps <= ONE_SLICE) {
    p.waves = 16;
    p.slices = 1;
    return p;
  }
  // one workgroup fits a compute unit, two where the sums of 16 rows are all it holds
  const int most = M <= 16 ? 512 : 256;
  p.slices = int(std::min<int64_t>(
      {(steps + 7) / 8, MAX_SLICES, std::max<int64_t>(1, most / p.blocks)}));
  return p;
}

// what a few-row kernel reads: dY; or dH, G, U of a gated pair with where dG and
// dU go; or a pair's dG and dU
struct Rows {
  const uint16_t *d, *G, *U;
  uint16_t *dG, *dU;
};

// 8 values of the pair's dG (layer 0) or dU (layer 1)
template <int ACT>
__device__ __forceinline__ uint4 pair_grad8(const uint4 h, const uint4 g, const uint4 u,
                                            int layer) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w},
                 uw[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a0, d0, a1, d1;
    gate_act_grad<ACT>(__uint_as_float(gw[j] << 16), a0, d0);
    gate_act_grad<ACT>(__uint_as_float(gw[j] & 0xFFFF0000u), a1, d1);
    const float h0 = __uint_as_float(hw[j] << 16), h1 = __uint_as_float(hw[j] & 0xFFFF0000u);
    const float u0 = __uint_as_float(uw[j] << 16), u1 = __uint_as_float(uw[j] & 0xFFFF0000u);
    o[j] = layer ? pack_bf16x2(h0 * a0, h1 * a1) : pack_bf16x2(h0 * u0 * d0, h1 * u1 * d1);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ACT >= 0: a gated pair, whose dG and dU every workgroup forms for itself (those
// of the first 128 columns store them); PLAIN_PAIR: a pair with dG and dU given;
// PLAIN: one layer
constexpr int PLAIN = -1, PLAIN_PAIR = -2;

template <int MT, int ACT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void grad_slice_kernel(Rows in, svdq::AwqWeight wa,
                                                                svdq::AwqWeight wb, int M, int K,
                                                                int N, int S, int sub,
                                                                float* __restrict__ part,
                                                                void* __restrict__ dX, bool xbf16) {
  constexpr int NT = 64 * WAVES;
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int LAYERS = ACT == PLAIN ? 1 : 2;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int slice = blockIdx.x % S, block = blockIdx.x / S;
  const int per = (N + 31) / 32, steps = per * LAYERS;
  const int s0 = int(int64_t(slice) * steps / S), s1 = int(int64_t(slice + 1) * steps / S);
  const int g = min(2 * block + (r >> 3), K / 64 - 1);

  v4f acc[MT][8];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[mt][t] = v4f{0, 0, 0, 0};

  struct Slot {
    uint32_t w[8];
    uint4 s, z;
  };
  // rows n past N (a multiple of 16) repeat the last ones; their scales are
  // cleared where they are used
  auto row8 = [&](int s) { return 32 * int64_t(s % per) + 8 * j; };
  auto fetch = [&](int s, Slot& sl) __attribute__((always_inline)) {
    const svdq::AwqWeight& w = LAYERS == 2 && s >= per ? wb : wa;
    const int64_t at = int64_t(g) * N + min(row8(s), int64_t(N) - 8);
    sl.s = *reinterpret_cast<const uint4*>(w.s + at);
    sl.z = *reinterpret_cast<const uint4*>(w.z + at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sl.w[i] = *reinterpret_cast<const uint32_t*>(w.q + (at + i) * 32 + 4 * (r & 7));
  };

  // `sub` steps of the rows' operand at a time in LDS, rows of 64 sub + 16 bytes
  const int rowb = sub * 64 + 16;
  int aoff[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) aoff[mt] = min(16 * mt + r, M - 1) * rowb + 16 * j;
  for (int c0 = s0; c0 < s1; c0 += sub) {
    const int here = min(sub, s1 - c0);
    if (c0 != s0) __syncthreads();
    Slot sl;
    if (wave < here) fetch(c0 + wave, sl);
    for (int i = tid; i < M * here * 4; i += NT) {
      const int m = i / (here * 4), o = i - m * (here * 4);
      const int s = c0 + (o >> 2), layer = LAYERS == 2 && s >= per;
      const int64_t n = 32 * int64_t(s - layer * per) + 8 * (o & 3), at = int64_t(m) * N + n;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (n < N) {
        const uint16_t* const d = ACT == PLAIN_PAIR ? (layer ? in.dU : in.dG) : in.d;
        v = *reinterpret_cast<const uint4*>(d + at);
        if constexpr (ACT >= 0) {
          const uint4 G = *reinterpret_cast<const uint4*>(in.G + at);
          const uint4 U = *reinterpret_cast<const uint4*>(in.U + at);
          v = pair_grad8<ACT>(v, G, U, layer);
          uint16_t* const out = layer ? in.dU : in.dG;
          if (block == 0) *reinterpret_cast<uint4*>(out + at) = v;
        }
      }
      *reinterpret_cast<uint4*>(lds + m * rowb + 16 * o) = v;
    }
    __syncthreads();
    for (int c = wave; c < here; c += WAVES) {
      const bool live = row8(c0 + c) < N;
      uint32_t o[8][4];
      const uint32_t sw[4] = {sl.s.x, sl.s.y, sl.s.z, sl.s.w};
      const uint32_t zw[4] = {sl.z.x, sl.z.y, sl.z.z, sl.z.w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float v[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float f = __uint_as_float(!live ? 0u : q ? sw[p] & 0xFFFF0000u : sw[p] << 16);
          const float zs = -__uint_as_float(q ? zw[p] & 0xFFFF0000u : zw[p] << 16) * f;
          dequant8_f32(sl.w[2 * p + q], f, zs, v[q]);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) o[t][p] = pack_bf16x2(v[0][t], v[1][t]);
      }
      if (c + WAVES < here) fetch(c0 + c + WAVES, sl);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const v8bf a = *reinterpret_cast<const v8bf*>(lds + aoff[mt] + 64 * c);
#pragma unroll
        for (int t = 0; t < 8; ++t)
          acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a, __builtin_bit_cast(v8bf, make_uint4(o[t][0], o[t][1], o[t][2], o[t][3])),
              acc[mt][t], 0, 0, 0);
      }
    }
  }

  // the waves' sums in order, one block of 16 rows at a time: thread (wave w,
  // lane) adds the eight sums of product w
  v4f* const red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 8; ++t) red[(t * WAVES + wave) * 64 + lane] = acc[mt][t];
    __syncthreads();
    if (wave >= 8) continue;
    v4f v = red[wave * WAVES * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[(wave * WAVES + w) * 64 + lane];
    const int64_t k = 128 * int64_t(block) + 64 * (r >> 3) + 8 * (r & 7) + wave;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t m = 16 * mt + 4 * j + e;
      if (m >= M || k >= K) continue;
      if (S > 1)
        part[(slice * int64_t(M) + m) * K + k] = v[e];
      else if (xbf16)
        static_cast<uint16_t*>(dX)[m * K + k] = f32_to_bf16(v[e]);
      else
        static_cast<float*>(dX)[m * K + k] = v[e];
    }
  }
}

// 4 columns per thread
__global__ __launch_bounds__(64) void grad_sum_kernel(const float* __restrict__ part, int S,
                                                      int64_t total, void* __restrict__ dX,
                                                      bool xbf16) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= total) return;
  // all loads first; a slice past the last counts as zeros
  v4f v[MAX_SLICES], p = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < MAX_SLICES; ++q)
    v[q] = reinterpret_cast<const v4f*>(part)[int64_t(min(q, S - 1)) * total + i];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int q = 0; q < MAX_SLICES; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] += q < S ? v[q][e] : 0.f;
  if (xbf16)
    static_cast<uint2*>(dX)[i] = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
  else
    static_cast<v4f*>(dX)[i] = p;
}

svdq_status launch_sum(const float* part, int S, int64_t M, int64_t K, void* dX, bool xbf16,
                       hipStream_t s) {
  const int64_t total = M * K / 4;
  hipLaunchKernelGGL(grad_sum_kernel, dim3(unsigned((total + 63) / 64)), dim3(64), 0, s, part, S,
                     total, dX, xbf16);
  return svdq::check_launch("grad_sum");
}

template <int MT, int ACT, int WAVES>
svdq_status run_slices(const Rows& in, int64_t M, int64_t K, int64_t N, const svdq::AwqWeight* w,
                       const Split& p, float* part, void* dX, bool xbf16, hipStream_t s) {
  constexpr int layers = ACT == PLAIN ? 1 : 2;
  // steps of the rows' operand that fit LDS (64 rows: 31)
  const int64_t steps = (N + 31) / 32 * layers;
  const int64_t room = MT == 1 ? LDS_A : 2 * LDS_A;
  const int sub = int(std::min<int64_t>((room / M - 16) / 64, (steps + p.slices - 1) / p.slices));
  const size_t shm = std::max(size_t(M) * (sub * 64 + 16), size_t(WAVES) * 8 * 1024);
  auto k = grad_slice_kernel<MT, ACT, WAVES>;
  // (the most that any call asks for: the attribute is the function's, and a host
  // thread with a smaller call must not lower it between another's two steps)
  static_assert(WAVES * 8 * 1024 <= 2 * LDS_A, "the sums fit");
  if (shm > (64 << 10))
    SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, 2 * LDS_A));
  hipLaunchKernelGGL(k, dim3(unsigned(p.blocks * p.slices)), dim3(64 * WAVES), shm, s, in, w[0],
                     w[layers - 1], int(M), int(K), int(N), p.slices, sub, part, dX, xbf16);
  return svdq::check_launch("grad_slice");
}

template <int ACT>
svdq_status run_rows(const Rows& in, int64_t M, int64_t K, int64_t N, const svdq::AwqWeight* w,
                     void* dX, bool xbf16, float* part, hipStream_t s) {
  const Split p = split(M, K, N, ACT == PLAIN ? 1 : 2);
  switch ((M + 15) / 16) {
    case 1:
      SVDQ_TRY(p.waves == 16 ? (run_slices<1, ACT, 16>(in, M, K, N, w, p, part, dX, xbf16, s))
                             : (run_slices<1, ACT, 8>(in, M, K, N, w, p, part, dX, xbf16, s)));
      break;
    case 2: SVDQ_TRY((run_slices<2, ACT, 8>(in, M, K, N, w, p, part, dX, xbf16, s))); break;
    case 3: SVDQ_TRY((run_slices<3, ACT, 8>(in, M, K, N, w, p, part, dX, xbf16, s))); break;
    default: SVDQ_TRY((run_slices<4, ACT, 8>(in, M, K, N, w, p, part, dX, xbf16, s))); break;
  }
  return p.slices == 1 ? SVDQ_OK : launch_sum(part, p.slices, M, K, dX, xbf16, s);
}

// ---------------------------------------------------------- many rows
// The weights are dequantized once into the workspace, transposed: row k holds
// the n of the first layer, then those of the second, each padded with zeros to a
// multiple of 64, in the blocks of gemm_bf16.h.

// 64 n (two stages) x 64 k (one group) per wave: lane (o, j) takes 8 rows n and 8
// k of each; through the wave's LDS every store then covers 16 rows k in a row
// (12288 x 4096: 129 MB in 24 us, 5.4 TB/s; stores of 64 bytes took 32)
__global__ __launch_bounds__(256) void transpose_dequant_kernel(svdq::AwqWeight w, int N,
                                                                int64_t stages, int64_t first,
                                                                uint16_t* __restrict__ B) {
  __shared__ uint4 lds[4][2][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int o = lane & 7, j = lane >> 3;
  const int blocks = ((N + 63) / 64 + 3) / 4, g = blockIdx.x / blocks;
  const int64_t n0 = int64_t(blockIdx.x % blocks) * 256 + 64 * wave;
  if (n0 >= (int64_t(N) + 63) / 64 * 64) return;
  const int64_t n = n0 + 8 * o;
  uint4 out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = make_uint4(0, 0, 0, 0);
  if (n < N) transpose_dequant8(w, int64_t(g) * N + n, j, out);
#pragma unroll
  for (int i = 0; i < 8; ++i) lds[wave][o >> 2][8 * j + i][o & 3] = out[i];
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 16 * i + (lane >> 2);
      *svdq_gemm::weight_at(B, stages, 64 * int64_t(g) + k, first + n0 + 32 * t + 8 * (lane & 3)) =
          lds[wave][t][k][lane & 3];
    }
}

__global__ __launch_bounds__(svdq_gemm::NT) void grad_wide_kernel(svdq_gemm::Args p,
                                                                  void* __restrict__ dX,
                                                                  bool xbf16) {
  using namespace svdq_gemm;
  __shared__ Stage st0, st1, st2, st3, st4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int64_t m0, b0;
  tile_origin((p.M + BM - 1) / BM, (p.rows + BN - 1) / BN, BM, BN, m0, b0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  tile_product(p, m0, b0, st0, st1, st2, st3, st4, acc);
  const int64_t row0 = m0 + (wave >> 2) * WM, col0 = b0 + (wave & 3) * WN;
  float* const eb = epilogue_buffer<32 * (WN + 4)>(wave, st0, st1, st2);
  const float none[CBL] = {0.f, 0.f};
  if (xbf16)
    store_wave_tile<RBL, CBL, true>(acc, none, eb, lane, row0, col0, p.M, p.rows, dX);
  else
    store_wave_tile<RBL, CBL, false>(acc, none, eb, lane, row0, col0, p.M, p.rows, dX);
}

// -------------------------------------------------------- medium number of rows
// B rows of a tile: 128 columns k of dX (two groups) over 64 n of one layer.
// A thread takes 4 rows n and 8 k of each, and writes 8 pieces of 4 n.  The
// swizzle has two more bits of the row than A's, so that the 8 k (rows 8 j + i)
// of 8 neighbouring threads fall into 8 different slots.
typedef float v8f __attribute__((ext_vector_type(8)));

struct GradWeights {
  svdq::AwqWeight wa, wb;
  int64_t gN;
  int N, chunks, j, quad, kr;
  uint32_t c[2][4];
  uint2 s2[2], z2[2];
  bool live[2];
  v8f even;
  v8i o0, o1;               // rows 0, 1 and rows 2, 3

  __device__ __forceinline__ GradWeights(const svdq::AwqWeight& a, const svdq::AwqWeight& b, int K,
                                         int N, int chunks, int64_t k0)
      : wa(a), wb(b), N(N), chunks(chunks) {
    const int t = threadIdx.x;
    j = t & 7;
    quad = (t >> 3) & 15;
    kr = 64 * (t >> 7) + 8 * j;
    gN = min(k0 / 64 + (t >> 7), int64_t(K) / 64 - 1) * N;
  }
  static __device__ __forceinline__ int slot(int row, int piece) {
    return row * 8 + (piece ^ (((row >> 1) ^ (row >> 4)) & 7));
  }
  template <int set>
  __device__ __forceinline__ void fetch(int chunk) {
    const bool second = chunk >= chunks;
    const uint8_t* const wq = second ? wb.q : wa.q;
    const uint16_t* const ws = second ? wb.s : wa.s;
    const uint16_t* const wz = second ? wb.z : wa.z;
    const int64_t n = 64 * int64_t(second ? chunk - chunks : chunk) + 4 * quad;
    live[set] = n < N;
    const int64_t at = gN + min(n, int64_t(N) - 4);
    s2[set] = *reinterpret_cast<const uint2*>(ws + at);
    z2[set] = *reinterpret_cast<const uint2*>(wz + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[set][i] = *reinterpret_cast<const uint32_t*>(wq + (at + i) * 32 + 4 * j);
  }
  // one row per quarter, packed in pairs; the last writes all four
  template <int set, int q>
  __device__ __forceinline__ void put(uint4* b) {
    const uint32_t sw = q < 2 ? s2[set].x : s2[set].y, zw = q < 2 ? z2[set].x : z2[set].y;
    const float f = __uint_as_float(!live[set] ? 0u : q & 1 ? sw & 0xFFFF0000u : sw << 16);
    float r[8];
    dequant8_f32(c[set][q], f, -__uint_as_float(q & 1 ? zw & 0xFFFF0000u : zw << 16) * f, r);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if constexpr (q == 1) o0[t] = int(pack_bf16x2(even[t], r[t]));
      if constexpr (q == 3) o1[t] = int(pack_bf16x2(even[t], r[t]));
      if constexpr (!(q & 1)) even[t] = r[t];
    }
    if constexpr (q == 3)
#pragma unroll
      for (int t = 0; t < 8; ++t)
        reinterpret_cast<uint2*>(b + slot(kr + t, quad >> 1))[quad & 1] =
            make_uint2(uint32_t(o0[t]), uint32_t(o1[t]));
  }
};

__global__ __launch_bounds__(svdq_mid::NT, 2) void grad_mid_kernel(
    svdq_mid::Args p, svdq::AwqWeight wa, svdq::AwqWeight wb, int K, int N, int S, int tiles,
    void* __restrict__ dX, bool xbf16, float* __restrict__ part) {
  using namespace svdq_mid;
  __shared__ ChunkA a0, a1, a2;
  __shared__ ChunkB b0, b1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = blockIdx.x / tiles;
  int64_t m0, k0;
  tile_at(int(blockIdx.x % tiles), (p.M + BM - 1) / BM, (K + BN - 1) / BN, BM, BN, m0, k0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  GradWeights w(wa, wb, K, N, p.chunks, k0);
  const int64_t total = int64_t(p.chunks) * p.segments;
  tile_product(p, m0, int(slice * total / S), int((slice + 1) * total / S), w, a0, a1, a2, b0, b1,
               acc);
  const int64_t row0 = m0 + (wave >> 1) * 64, col0 = k0 + (wave & 1) * 64;
  float* const eb = reinterpret_cast<float*>(wave == 0   ? &a0.v
                                              : wave == 1 ? &a1.v
                                              : wave == 2 ? &a2.v
                                                          : &b0.v);
  const float none[CBL] = {0.f, 0.f};
  if (S > 1)
    store_wave_tile<RBL, CBL, false>(acc, none, eb, lane, row0, col0, p.M, K,
                                     part + int64_t(slice) * p.M * K);
  else if (xbf16)
    store_wave_tile<RBL, CBL, true>(acc, none, eb, lane, row0, col0, p.M, K, dX);
  else
    store_wave_tile<RBL, CBL, false>(acc, none, eb, lane, row0, col0, p.M, K, dX);
}

int mid_slices(int64_t M, int64_t K, int64_t N, int layers) {
  return svdq_mid::slices((M + 127) / 128 * ((K + 127) / 128), (N + 63) / 64 * layers);
}

// dX = A0 wd0 [+ A1 wd1]
svdq_status launch_mid(const uint16_t* A0, const uint16_t* A1, const svdq::AwqWeight* w,
                       int layers, int64_t M, int64_t K, int64_t N, void* dX, bool xbf16,
                       float* part, hipStream_t s) {
  const int64_t tiles = (M + 127) / 128 * ((K + 127) / 128);
  const int S = mid_slices(M, K, N, layers);
  svdq_mid::Args p{{A0, A1}, N, int((N + 63) / 64), layers, int(M)};
  hipLaunchKernelGGL(grad_mid_kernel, dim3(unsigned(tiles * S)), dim3(svdq_mid::NT), 0, s, p, w[0],
                     w[layers - 1], int(K), int(N), S, int(tiles), dX, xbf16, part);
  SVDQ_TRY(svdq::check_launch("awq_grad (mid)"));
  return S == 1 ? SVDQ_OK : launch_sum(part, S, M, K, dX, xbf16, s);
}

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

int64_t wide_rows(int64_t M, int64_t K, int64_t N, int layers) {
  if (M <= ROWS) return 0;
  return svdq_plan::wide_rows(
      M, {pad64(N) / 64 * layers, (K + 255) / 256, (K + 127) / 128, layers * K * N});
}

size_t transposed_bytes(int64_t K, int64_t N, int layers) {
  return svdq_gemm::weight_bytes(K, pad64(N) / 32 * layers);
}

// bytes of the partial sums of `rows` rows
size_t part_bytes(int64_t rows, int64_t K, int64_t N, int layers) {
  if (rows == 0) return 0;
  const int S = rows <= ROWS ? split(rows, K, N, layers).slices : mid_slices(rows, K, N, layers);
  return S == 1 ? 0 : svdq::align256(size_t(S) * size_t(rows) * size_t(K) * 4);
}

// dX = A0 wd0 [+ A1 wd1], B the workspace
svdq_status launch_wide(const uint16_t* A0, const uint16_t* A1, const svdq::AwqWeight* w,
                        int layers, int64_t M, int64_t K, int64_t N, void* dX, bool xbf16,
                        uint16_t* B, hipStream_t s) {
  const int64_t np = pad64(N);
  for (int i = 0; i < layers; ++i) {
    hipLaunchKernelGGL(transpose_dequant_kernel, dim3(unsigned((np + 255) / 256 * (K / 64))),
                       dim3(256), 0, s, w[i], int(N), np / 32 * layers, i * np, B);
    SVDQ_TRY(svdq::check_launch("transpose_dequant"));
  }
  svdq_gemm::Args p{{A0, A1}, N, int(np / 64), layers, B, int(M), int(K)};
  const int64_t tiles = ((M + 255) / 256) * ((K + 255) / 256);
  hipLaunchKernelGGL(grad_wide_kernel, dim3(unsigned(tiles)), dim3(svdq_gemm::NT), 0, s, p, dX,
                     xbf16);
  return svdq::check_launch("grad_wide");
}

}  // namespace

namespace svdq {

size_t awq_linear_grad_workspace(int64_t M, int64_t K, int64_t N) {
  const int64_t w = wide_rows(M, K, N, 1);
  return (w ? transposed_bytes(K, N, 1) : 0) + part_bytes(M - w, K, N, 1);
}

size_t awq_gated_grad_workspace(int64_t M, int64_t K, int64_t N) {
  const int64_t w = wide_rows(M, K, N, 2);
  return (w ? transposed_bytes(K, N, 2) : 0) + part_bytes(M - w, K, N, 2);
}

svdq_status launch_awq_linear_grad(const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                                   AwqWeight wt, void* dX, svdq_dtype x_dt, void* ws,
                                   hipStream_t s) {
  const int64_t w = wide_rows(M, K, N, 1), rest = M - w;
  const bool xb = x_dt == SVDQ_BF16;
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  if (w) SVDQ_TRY(launch_wide(dY, dY, &wt, 1, w, K, N, dX, xb, reinterpret_cast<uint16_t*>(w8), s));
  if (!rest) return SVDQ_OK;
  float* const part = reinterpret_cast<float*>(w8 + (w ? transposed_bytes(K, N, 1) : 0));
  const uint16_t* const d = dY + w * N;
  void* const x = static_cast<uint8_t*>(dX) + w * K * (xb ? 2 : 4);
  const Rows in{d, nullptr, nullptr, nullptr, nullptr};
  if (rest <= ROWS) return run_rows<PLAIN>(in, rest, K, N, &wt, x, xb, part, s);
  return launch_mid(d, d, &wt, 1, rest, K, N, x, xb, part, s);
}

svdq_status launch_awq_gated_grad(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                  int64_t M, int64_t K, int64_t N, AwqWeight wg, AwqWeight wu,
                                  svdq_act act, uint16_t* dX, uint16_t* dG, uint16_t* dU, void* ws,
                                  hipStream_t s) {
  const AwqWeight wt[2] = {wg, wu};
  const int64_t w = wide_rows(M, K, N, 2), rest = M - w;
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  float* const part = reinterpret_cast<float*>(w8 + (w ? transposed_bytes(K, N, 2) : 0));
  // few rows form their own dG and dU unless too many columns of dX repeat that
  const bool fused = rest <= ROWS && rest * N <= FUSED_GRADS / ((K + 127) / 128);
  const Rows in{dH + w * N, G + w * N, U + w * N, dG + w * N, dU + w * N};
  uint16_t* const x = dX + w * K;
  if (rest && fused)
    SVDQ_TRY(act == SVDQ_SILU ? run_rows<SVDQ_SILU>(in, rest, K, N, wt, x, true, part, s)
                              : run_rows<SVDQ_GELU>(in, rest, K, N, wt, x, true, part, s));
  const int64_t tiled = fused ? w : M;
  if (!tiled) return SVDQ_OK;
  const int64_t n8 = tiled * N / 8;
  const unsigned blocks = unsigned(std::min<int64_t>((n8 + 255) / 256, 16384));
  auto k = act == SVDQ_SILU ? gate_grad_kernel<SVDQ_SILU> : gate_grad_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(blocks), dim3(256), 0, s, dH, G, U, n8, dG, dU);
  SVDQ_TRY(check_launch("gate_grad"));
  if (w)
    SVDQ_TRY(launch_wide(dG, dU, wt, 2, w, K, N, dX, true, reinterpret_cast<uint16_t*>(w8), s));
  if (!rest || fused) return SVDQ_OK;
  if (rest <= ROWS) return run_rows<PLAIN_PAIR>(in, rest, K, N, wt, x, true, part, s);
  return launch_mid(in.dG, in.dU, wt, 2, rest, K, N, x, true, part, s);
}

}  // namespace svdq
