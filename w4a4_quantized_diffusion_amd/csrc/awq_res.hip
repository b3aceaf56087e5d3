// AWQ W4A16 product with bias, activation, gate and residual in its epilogue (gfx950):
//
//   Z = X wd^T + bias,   Y = R + gate * act(Z)
//
// wd = bf16((q - z) s) [N, K], X bf16 [M, K], gate one vector of N for all rows or one
// per image, R [M, N] fp32 or bf16.  Z stays in the fp32 accumulators of the bf16
// MFMAs; Y is rounded once.  Z can be stored in bf16 for the backward pass
//
//   dZ = dY * gate * act'(Z),  dX = dZ wd,  dgate = sum over rows of dY * act(Z)
//
// whose first and last part are here, the product in awq_grad.hip.

#include "block.h"
#include "gemm_bf16.h"

using namespace svdq_dev;

namespace {

using svdq::ResEpilogue;

template <int ACT>
__device__ __forceinline__ float act_of(float x) {
  if constexpr (ACT == SVDQ_NO_ACT) {
    return x;
  } else if constexpr (ACT == SVDQ_GELU) {
    // x / (1 + exp2(x (c1 + c3 x^2))): gate_act's argument in three operations instead of
    // seven (4608 rows 4096 -> 12288: 434.6 us for 438.1, 0.8%)
    constexpr float c1 = -1.5957691216057308f * LOG2E, c3 = 0.044715f * c1;
    return x * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * fmaf(c3, x * x, c1)));
  } else {
    return gate_act<ACT>(x);
  }
}

// V values at any address that is a multiple of their size (a copy leaves the compiler
// to choose loads that the target takes there)
template <int V>
__device__ __forceinline__ void load_any(const void* p, bool b16, int64_t at, float (&v)[V]) {
  if (b16) {
    uint16_t t[V];
    __builtin_memcpy(t, static_cast<const uint16_t*>(p) + at, 2 * V);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = bf16_to_f32(t[i]);
  } else {
    __builtin_memcpy(v, static_cast<const float*>(p) + at, 4 * V);
  }
}

__device__ __forceinline__ int64_t gate_at(const ResEpilogue& e, int m, int64_t n) {
  return (e.gate.ld ? e.gate.ld * (uint32_t(e.first + m) / uint32_t(e.rows)) : 0) + n;
}

// V (4 or 8) neighbouring outputs of row m from column n on: z = acc + bias
// (Non-temporal stores: many rows alone 1-10% faster, 4300 rows 1024 -> 4096 60.5 us for 67,
// and blocks of norm and products one behind the other as fast as with ordinary ones.)
template <int ACT, int V>
__device__ __forceinline__ void emit(const ResEpilogue& e, int m, int64_t n, int64_t N,
                                     float (&z)[V]) {
  const int64_t at = int64_t(m) * N + n;
  auto put = [&](void* Y, bool b16, const float (&v)[V]) __attribute__((always_inline)) {
    if (b16) {
      uint16_t* const p = static_cast<uint16_t*>(Y) + at;
      if constexpr (V == 8)
        __builtin_nontemporal_store(
            v4i{int(pack_bf16x2(v[0], v[1])), int(pack_bf16x2(v[2], v[3])),
                int(pack_bf16x2(v[4], v[5])), int(pack_bf16x2(v[6], v[7]))},
            reinterpret_cast<v4i*>(p));
      else
        *reinterpret_cast<uint2*>(p) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
      float* const p = static_cast<float*>(Y) + at;
#pragma unroll
      for (int i = 0; i < V; i += 4)
        __builtin_nontemporal_store(v4f{v[i], v[i + 1], v[i + 2], v[i + 3]},
                                    reinterpret_cast<v4f*>(p + i));
    }
  };
  if (e.Z) put(e.Z, true, z);
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = act_of<ACT>(z[i]);
  if (e.gate.p) {
    float g[V];
    load_any<V>(e.gate.p, e.gate.b16, gate_at(e, m, n), g);
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] *= g[i];
  }
  if (e.R) {
    float r[V];
    load_any<V>(e.R, e.r16, at, r);
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] += r[i];
  }
  put(e.Y, e.y16, z);
}

// A wave's RBL x CBL blocks of 32 x 32 in the accumulators, through its LDS buffer
// `eb` (32 x (32 CBL + 4) floats), so that a lane has 8 neighbouring columns of a row.
template <int ACT, int RBL, int CBL>
__device__ __forceinline__ void res_epilogue(const ResEpilogue& e, const v16f (&acc)[RBL][CBL],
                                             float* eb, int lane, int64_t row0, int64_t col0,
                                             int M, int N) {
  constexpr int ER = 32 * CBL + 4, CH = 4 * CBL, RPI = 64 / CH;
  const int h = lane >> 5, r32 = lane & 31, q = lane % CH;
  const int64_t n = col0 + 8 * q;
  float b[8] = {};
  if (e.bias && n < N) load_any<8>(e.bias, true, n, b);
#pragma unroll
  for (int i = 0; i < RBL; ++i) {
#pragma unroll
    for (int j = 0; j < CBL; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k)
        eb[(8 * (k >> 2) + 4 * h + (k & 3)) * ER + j * 32 + r32] = acc[i][j][k];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int t = 0; t < 32 / RPI; ++t) {
      const int rr = lane / CH + RPI * t;
      const float4 u = *reinterpret_cast<const float4*>(eb + rr * ER + 8 * q);
      const float4 v = *reinterpret_cast<const float4*>(eb + rr * ER + 8 * q + 4);
      const int64_t m = row0 + i * 32 + rr;
      float z[8] = {u.x + b[0], u.y + b[1], u.z + b[2], u.w + b[3],
                    v.x + b[4], v.y + b[5], v.z + b[6], v.w + b[7]};
      if (m < M && n < N) emit<ACT, 8>(e, int(m), n, N, z);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ----------------------------------------------------------- few rows
// Up to 64 rows the time is the weights' way from memory and how many launches follow
// one another.  One launch where X is small (res_column_kernel), else slices of K
// whose partial sums a second launch joins with the epilogue.

constexpr int ROWS = 64;
constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int LDS_X = 64 << 10;
constexpr int SUM_SLICES = 8;

struct Split {
  int blocks, slices;
};

// Up to 8 slices, as many as the second launch loads at once, and up to 16 of at least
// eight chunks each: 64 rows 16384 -> 4096 32.7 -> 24.5 us, 17 rows 8192 -> 512 10.2 -> 8.7;
// with slices of four chunks 33 rows 4096 -> 4096 take 12.5 us instead of 11.4.
Split split(int64_t M, int64_t K, int64_t N) {
  Split p;
  p.blocks = int((N + 16 * WAVES - 1) / (16 * WAVES));
  p.slices = int(std::min<int64_t>(
      {K / 64, std::max<int64_t>(SUM_SLICES, std::min<int64_t>(16, K / 512)),
       std::max<int64_t>(1, 512 / p.blocks)}));
  return p;
}

// Whether few rows take one launch, where every 16 columns read all of X from the L2 (2 M
// K N / 16 bytes) and a wave's rows of X grow with M K.  Measured, one launch against two,
// us: 2048 -> 2048 1 row 3.8 / 6.1, 48 rows 8.4 / 8.9, 64 rows 10.3 / 9.8; 4096 -> 4096 24
// rows 9.7 / 10.4, 33 rows 15.2 / 11.2; 2048 -> 8192 24 rows 9.8 / 10.5, 33 rows 12.5 /
// 11.9; 8192 -> 2048 8 rows 9.3 / 9.2, 12 rows 10.6 / 9.3; 4096 -> 12288 8 rows 12.4 /
// 13.9, 16 rows 16.3 / 14.6, 64 rows 48 / 23.5; 12288 -> 4096 8 rows 12.3 / 13.1, 12 rows
// 13.3 / 13.2.
bool one_launch(int64_t M, int64_t K, int64_t N) {
  return M * K <= 3 << 15 && M * K <= (27 << 24) / N;
}

// One chunk of 64 k of 16 rows of the weights: lane group j holds the codes
// k = 16 j .. 16 j + 15 of its row.
struct Codes {
  uint2 w;
  uint32_t s, z;
};

__device__ __forceinline__ void fetch_codes(Codes& c, const svdq::AwqWeight& w, int64_t at, int j) {
  c.w = *reinterpret_cast<const uint2*>(w.q + at * 32 + 8 * j);
  c.s = w.s[at];
  c.z = w.z[at];
}

// past the last chunk (not live) the scales are zeros
__device__ __forceinline__ void operands(const Codes& c, bool live, v8bf (&b)[2]) {
  const float s = live ? __uint_as_float(c.s << 16) : 0.f;
  const float zs = -__uint_as_float(c.z << 16) * s;
  b[0] = __builtin_bit_cast(v8bf, dequant8(c.w.x, s, zs));
  b[1] = __builtin_bit_cast(v8bf, dequant8(c.w.y, s, zs));
}

// A workgroup's 8 waves take 16 columns each and one of S slices of K, whose part of X they
// share in LDS; a wave's weights are four chunks ahead in registers.  64 rows 4096 -> 12288
// take 23 us with the second launch: 28 MB of weights, and 16 MB of partial sums written
// and read, 2.7 TB/s, half of a copy's rate; 16 rows 14.5.  Not memory: a piece of X is
// loaded, written to LDS, waited for and multiplied before the next one begins.  LDS_X holds
// 8 chunks of up to 63 rows and 4 of 64, which then take twice the pieces: 63 and 64 rows
// 4096 -> 12288 22.5-23.1 and 22.6-23.0 us, 4096 -> 4096 14.7 and 15.4.
template <int MT>
__global__ __launch_bounds__(NT, 4) void res_slice_kernel(const uint16_t* __restrict__ X, int M,
                                                          int K, int N, svdq::AwqWeight w, int S,
                                                          int sub, float* __restrict__ part) {
  constexpr int D = 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int G = K / 64;
  const int slice = blockIdx.x % S;
  const int g0 = int(int64_t(slice) * G / S), count = int(int64_t(slice + 1) * G / S) - g0;
  const int64_t n = (int64_t(blockIdx.x / S) * WAVES + wave) * 16 + r;
  const int64_t nc = min(n, int64_t(N) - 1);
  Codes ring[D];
  // every slot is always loaded (past the last chunk with the last one's data), so that
  // the number of loads in flight is fixed
  auto fetch = [&](int i, Codes& c) __attribute__((always_inline)) {
    fetch_codes(c, w, int64_t(g0 + min(i, count - 1)) * N + nc, j);
  };
  v4f acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) acc[mt] = v4f{0, 0, 0, 0};
  // `sub` chunks of X at a time in LDS: rows of `sub` chunks and 16 bytes, so that 16
  // rows start in 16 different groups of 4 banks
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
        v8bf b[2];
        operands(ring[d], c + d < here, b);
        const uint8_t* const xc = lds + 128 * min(c + d, here - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                *reinterpret_cast<const v8bf*>(xc + xoff[mt] + 16 * h), b[h], acc[mt], 0, 0, 0);
        fetch(c0 + c + d + D, ring[d]);
      }
  }
  if (n >= N) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = 16 * mt + 4 * j + e;
      // (read by the next launch, on any XCD: past this one's L2 at once)
      if (m < M)
        __builtin_nontemporal_store(acc[mt][e], part + (int64_t(slice) * M + m) * N + n);
    }
}

// 4 columns per thread
template <int ACT>
__global__ __launch_bounds__(64) void res_sum_kernel(const float* __restrict__ part, int S, int M,
                                                     int N, ResEpilogue e) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x, total = int64_t(M) * N / 4;
  if (i >= total) return;
  const int64_t m = 4 * i / N, n = 4 * i - m * N;
  float z[4] = {}, b[4] = {};
  for (int q0 = 0; q0 < S; q0 += SUM_SLICES) {
    // all loads first; a slice past the last counts as zeros
    v4f v[SUM_SLICES];
#pragma unroll
    for (int q = 0; q < SUM_SLICES; ++q)
      v[q] = reinterpret_cast<const v4f*>(part)[int64_t(min(q0 + q, S - 1)) * total + i];
    __builtin_amdgcn_sched_barrier(0);
    if (q0 == 0 && e.bias) load_any<4>(e.bias, true, n, b);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int q = 0; q < SUM_SLICES; ++q) z[k] += q0 + q < S ? v[q][k] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) z[k] += b[k];
  emit<ACT, 4>(e, int(m), n, N, z);
}

// One launch: a workgroup owns 16 columns, its 8 waves take the chunks of K in turn,
// each with its own piece of X, and the sums meet in LDS.  One row 4096 -> 4096 5.4 us, 9 MB
// of weights at 1.7 TB/s: one workgroup a compute unit, two turns of four chunks a wave, a
// reduction and the epilogue, one after the other.
template <int MT, int ACT>
__global__ __launch_bounds__(NT, 4) void res_column_kernel(const uint16_t* __restrict__ X, int M,
                                                           int K, int N, svdq::AwqWeight w,
                                                           ResEpilogue e) {
  constexpr int D = MT == 1 ? 4 : 2;
  __shared__ v4f red[WAVES][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int64_t n = int64_t(blockIdx.x) * 16 + r;                   // (N is a multiple of 16)
  const int G = K / 64, count = (G - wave + WAVES - 1) / WAVES;     // chunks of this wave
  const uint16_t* xrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xrow[mt] = X + int64_t(min(16 * mt + r, M - 1)) * K + 16 * j;
  struct Slot {
    Codes c;
    uint4 x[MT][2];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's
  // data; a wave without chunks loads chunk 0 and never uses it)
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int c = count > 0 ? wave + WAVES * min(i, count - 1) : 0;
    fetch_codes(sl.c, w, int64_t(c) * N + n, j);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4* const x = reinterpret_cast<const uint4*>(xrow[mt] + 64 * int64_t(c));
      sl.x[mt][0] = x[0];
      sl.x[mt][1] = x[1];
    }
  };
  v4f acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) acc[mt] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, ring[d]);
  for (int c = 0; c < count; c += D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Slot& sl = ring[d];
      v8bf b[2];
      operands(sl.c, c + d < count, b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, sl.x[mt][h]),
                                                            b[h], acc[mt], 0, 0, 0);
      fetch(c + d + D, sl);
    }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) red[wave][mt][lane] = acc[mt];
  __syncthreads();
  // thread (wave w < MT, row t of its 16, columns 4 q ..): the sums from LDS, where
  // element (row 4 j + e, column r) lies in component e of lane 16 j + r
  if (wave >= MT) return;
  const int row = lane >> 2, q = lane & 3, m = 16 * wave + row;
  if (m >= M) return;
  float z[4], b[4] = {};
  const int64_t n0 = int64_t(blockIdx.x) * 16 + 4 * q;
  if (e.bias) load_any<4>(e.bias, true, n0, b);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int from = 16 * (row >> 2) + 4 * q + k;
    z[k] = reinterpret_cast<const float*>(&red[0][wave][from])[row & 3];
#pragma unroll
    for (int v = 1; v < WAVES; ++v)
      z[k] += reinterpret_cast<const float*>(&red[v][wave][from])[row & 3];
    z[k] += b[k];
  }
  emit<ACT, 4>(e, m, n0, N, z);
}

// ---------------------------------------------------------- many rows
// The weights dequantized once into the workspace: 64 rows and two groups of 64 k (two
// stages each) per workgroup; four lanes take one row, 8 k of each stage, so that a wave
// stores 1 KB in a row.  Neighbouring workgroups go along K: a row block's stages are
// consecutive in the workspace, while the same stage of other row blocks lies whole rows
// of stages apart, in the same memory channels (12288 x 4096: 129 MB in 22.8 us, 5.7
// TB/s; in the order of the rows 33).
constexpr int DEQUANT_GROUPS = 2;

__global__ __launch_bounds__(256) void res_dequant_kernel(svdq::AwqWeight w, int K, int N,
                                                          uint16_t* __restrict__ B) {
  const int row = threadIdx.x >> 2, piece = threadIdx.x & 3;
  const int G = K / 64, along = (G + DEQUANT_GROUPS - 1) / DEQUANT_GROUPS;
  const int g0 = blockIdx.x % along * DEQUANT_GROUPS;
  const int64_t n = int64_t(blockIdx.x / along) * 64 + row;
  if (n >= N) return;
  uint32_t c[DEQUANT_GROUPS][2];
  uint16_t s[DEQUANT_GROUPS], z[DEQUANT_GROUPS];
#pragma unroll
  for (int i = 0; i < DEQUANT_GROUPS; ++i) {
    const int64_t at = int64_t(min(g0 + i, G - 1)) * N + n;
    const uint32_t* const p = reinterpret_cast<const uint32_t*>(w.q + at * 32 + piece * 4);
    c[i][0] = p[0];
    c[i][1] = p[4];
    s[i] = w.s[at];
    z[i] = w.z[at];
  }
#pragma unroll
  for (int i = 0; i < DEQUANT_GROUPS; ++i) {
    if (g0 + i >= G) break;
    const float f = bf16_to_f32(s[i]), fz = -bf16_to_f32(z[i]) * f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      *svdq_gemm::weight_at(B, K / 32, n, 64 * (g0 + i) + 32 * t + 8 * piece) =
          dequant8(c[i][t], f, fz);
  }
}

template <int ACT>
__global__ __launch_bounds__(svdq_gemm::NT) void res_wide_kernel(svdq_gemm::Args p, ResEpilogue e) {
  using namespace svdq_gemm;
  __shared__ Stage st0, st1, st2, st3, st4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t m0, b0;
  tile_origin((p.M + BM - 1) / BM, (p.rows + BN - 1) / BN, BM, BN, m0, b0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  tile_product(p, m0, b0, st0, st1, st2, st3, st4, acc);
  res_epilogue<ACT, RBL, CBL>(e, acc, epilogue_buffer<32 * (WN + 4)>(wave, st0, st1, st2), lane,
                              m0 + (wave >> 2) * WM, b0 + (wave & 3) * WN, p.M, p.rows);
}

// Power bounds it as it does the plain product: 4608 rows 4096 -> 12288 in 390-440 us on
// different cards, 1.05-1.19 PFLOP/s, where the library's product of the shape has 1.30; the
// last 0.4 of a round is spread over all compute units (in whole tiles the call takes 15 us
// more).  Of that 28 us are the epilogues with GELU and Z stored, 8 us a tile of exp,
// reciprocal, conversions and stores that no other workgroup of the compute unit covers.
template <int ACT>
__global__ __launch_bounds__(svdq_gemm::NT) void res_split_kernel(svdq_gemm::Args p, ResEpilogue e,
                                                                  int64_t full, int S,
                                                                  float* __restrict__ part) {
  using namespace svdq_gemm;
  __shared__ Stage st0, st1, st2, st3, st4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Work w = work_of(p, full, S);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  tile_product(p, w.m0, w.b0, st0, st1, st2, st3, st4, acc, w.first, w.count);
  const int64_t row = (wave >> 2) * WM, col = (wave & 3) * WN;
  float* const eb = epilogue_buffer<32 * (WN + 4)>(wave, st0, st1, st2);
  if (w.split < 0) {
    res_epilogue<ACT, RBL, CBL>(e, acc, eb, lane, w.m0 + row, w.b0 + col, p.M, p.rows);
  } else {
    const float none[CBL] = {0.f, 0.f};
    store_wave_tile<RBL, CBL, false>(acc, none, eb, lane, row, col, BM, BN, part + w.split * TILE);
  }
}

// The split tiles' sums and the epilogue: a workgroup takes 8 rows of a tile, a thread 8
// columns of one.  96 tiles in two parts: 50 MB read, 25 MB of outputs, 15-17 us.
template <int ACT>
__global__ __launch_bounds__(256) void res_join_kernel(const float* __restrict__ part, int S,
                                                       int64_t full, int M, int N, ResEpilogue e) {
  const int tile = blockIdx.x >> 5, row = (blockIdx.x & 31) * 8 + (threadIdx.x >> 5);
  const int col = (threadIdx.x & 31) * 8;
  int64_t m0, n0;
  svdq_gemm::tile_of(full + tile, (M + 255) / 256, (N + 255) / 256, m0, n0);
  const int64_t m = m0 + row, n = n0 + col;
  if (m >= M || n >= N) return;
  const float* const p = part + int64_t(tile) * S * svdq_gemm::TILE + row * 256 + col;
  float z[8] = {};
  // (two slices' loads at a time; one past the last counts as zeros)
  for (int q = 0; q < S; q += 2) {
    v4f v[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[k][i] = reinterpret_cast<const v4f*>(p + min(q + k, S - 1) * svdq_gemm::TILE)[i];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += q + k < S ? v[k][i >> 2][i & 3] : 0.f;
  }
  if (e.bias) {
    float b[8];
    load_any<8>(e.bias, true, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
  }
  emit<ACT, 8>(e, int(m), n, N, z);
}

// -------------------------------------------------------- medium number of rows
// B rows of a tile: 128 rows of the weights, two threads to a row, 32 codes each.
struct RowWeights {
  // this thread's row of chunk 0; a chunk further is N rows further
  const uint8_t* q;
  const uint16_t *s, *z;
  int N, row, half;
  uint4 c[2];
  uint16_t cs[2], cz[2];

  __device__ __forceinline__ RowWeights(const svdq::AwqWeight& w, int N, int64_t n0,
                                        int tid = int(threadIdx.x))
      : N(N), row(tid >> 1), half(tid & 1) {
    const int64_t nr = min(n0 + row, int64_t(N) - 1);
    q = w.q + nr * 32 + 16 * half;
    s = w.s + nr;
    z = w.z + nr;
  }
  // (any 16 rows' pieces lie in different groups of 4 banks, which the reads need, and of
  // the eight of a cycle's writes, four rows and two pieces apart by 4, none is 8 slots
  // from another: with piece ^ (row / 2) a write took twice its cycles, the call 1-2% more)
  static __device__ __forceinline__ int slot(int row, int piece) {
    return row * 8 + (piece ^ (((row >> 1) ^ (2 * row & 2)) & 7));
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

// One set of four waves a tile (svdq_plan::medium says when): 333 rows 4096 -> 4096 28.3 us
// with the sums (0.39 PFLOP/s).
template <int ACT>
__global__ __launch_bounds__(svdq_mid::NT, 2) void res_mid_kernel(svdq_mid::Args p,
                                                                  svdq::AwqWeight wt, int N, int S,
                                                                  int tiles, ResEpilogue e,
                                                                  float* __restrict__ part) {
  using namespace svdq_mid;
  __shared__ ChunkA a0, a1, a2;
  __shared__ ChunkB b0, b1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = blockIdx.x / tiles;
  int64_t m0, n0;
  tile_at(int(blockIdx.x % tiles), (p.M + BM - 1) / BM, (N + BN - 1) / BN, BM, BN, m0, n0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  RowWeights w(wt, N, n0);
  tile_product(p, m0, int(int64_t(slice) * p.chunks / S), int(int64_t(slice + 1) * p.chunks / S), w,
               a0, a1, a2, b0, b1, acc);
  const int64_t row0 = m0 + (wave >> 1) * 64, col0 = n0 + (wave & 1) * 64;
  // 32 x 68 floats, in an LDS object of the wave's own
  float* const eb = reinterpret_cast<float*>(wave == 0   ? &a0.v
                                              : wave == 1 ? &a1.v
                                              : wave == 2 ? &a2.v
                                                          : &b0.v);
  if (S == 1) {
    res_epilogue<ACT, RBL, CBL>(e, acc, eb, lane, row0, col0, p.M, N);
    return;
  }
  const float none[CBL] = {0.f, 0.f};
  store_wave_tile<RBL, CBL, false>(acc, none, eb, lane, row0, col0, p.M, N,
                                   part + int64_t(slice) * p.M * N);
}

// The same tile by two such sets of four waves, each with half of a slice's chunks and LDS
// of its own.  333 rows 8192 -> 2064 in 5 slices of 51 tiles: 22-24 us (0.47-0.51 PFLOP/s)
// and 5 for the sums; one set a workgroup in 8 slices took 25 and 6.  Copies of the loop
// that only load take 13 us less the sums, and without the dequantization, the MFMAs or the LDS
// reads alone 6, 5 and 4 less: loads, vector, matrix and LDS work share a SIMD's two waves
// without hiding one another fully.  Runs of tiles for each XCD gain 5% at some sizes and
// cost 15% at others.
template <int ACT>
__global__ __launch_bounds__(2 * svdq_mid::NT, 2) void res_twin_kernel(svdq_mid::Args p,
                                                                       svdq::AwqWeight wt, int N,
                                                                       int S, int tiles,
                                                                       ResEpilogue e,
                                                                       float* __restrict__ part) {
  using namespace svdq_mid;
  __shared__ ChunkA a0[2], a1[2], a2[2];
  __shared__ ChunkB b0[2], b1[2];
  const int lane = threadIdx.x & 63, tid = threadIdx.x & (svdq_mid::NT - 1);
  const int half = __builtin_amdgcn_readfirstlane(threadIdx.x / svdq_mid::NT);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = blockIdx.x / tiles;
  int64_t m0, n0;
  tile_at(int(blockIdx.x % tiles), (p.M + BM - 1) / BM, (N + BN - 1) / BN, BM, BN, m0, n0);
  v16f acc[RBL][CBL], sum[1][CBL];
  zero_acc(acc);
  RowWeights w(wt, N, n0, tid);
  const int c0 = int(int64_t(slice) * p.chunks / S), c2 = int(int64_t(slice + 1) * p.chunks / S);
  const int c1 = (c0 + c2 + 1) / 2;
  tile_product(p, m0, half ? c1 : c0, half ? c2 : c1, w, a0[half], a1[half], a2[half], b0[half],
               b1[half], acc, tid);
  // a barrier a chunk, which the half with one chunk less makes up for
  if (half && c2 - c1 < c1 - c0) __builtin_amdgcn_s_barrier();
  add_halves(acc, half, wave, lane, b0, b1, sum);
  const int64_t row0 = m0 + (wave >> 1) * 64 + 32 * half, col0 = n0 + (wave & 1) * 64;
  // 32 x 68 floats, in an LDS object of the wave's own
  __syncthreads();
  float* const eb = reinterpret_cast<float*>(wave == 0   ? &a0[half].v
                                              : wave == 1 ? &a1[half].v
                                              : wave == 2 ? &a2[half].v
                                                          : &b0[half].v);
  if (S == 1) {
    res_epilogue<ACT, 1, CBL>(e, sum, eb, lane, row0, col0, p.M, N);
    return;
  }
  const float none[CBL] = {0.f, 0.f};
  store_wave_tile<1, CBL, false>(sum, none, eb, lane, row0, col0, p.M, N,
                                 part + int64_t(slice) * p.M * N);
}

int64_t mid_tiles(int64_t M, int64_t N) { return (M + 127) / 128 * ((N + 127) / 128); }

svdq_plan::Shape shape_of(int64_t K, int64_t N) {
  return {K / 64, (N + 255) / 256, (N + 127) / 128, K * N, true};
}

// the rows of the wide form, and whether its last round is split (then they are all)
int64_t wide_rows(int64_t M, int64_t K, int64_t N, svdq_gemm::Rounds* split) {
  split->S = 1;
  if (M <= ROWS) return 0;
  const svdq_plan::Shape shape = shape_of(K, N);
  double us;
  const int64_t w = svdq_plan::wide_rows(M, shape, &us);
  const svdq_gemm::Rounds r = svdq_gemm::rounds(M, N, K / 32);
  if (r.S == 1 || svdq_plan::split_us(r, shape) >= us) return w;
  *split = r;
  return M;
}

size_t weight_bytes(int64_t K, int64_t N) { return svdq_gemm::weight_bytes(N, K / 32); }

// bytes of the partial sums of `rows` rows
size_t part_bytes(int64_t rows, int64_t K, int64_t N) {
  if (rows == 0 || (rows <= ROWS && one_launch(rows, K, N))) return 0;
  const int S = rows <= ROWS ? split(rows, K, N).slices
                             : svdq_plan::medium(rows, shape_of(K, N)).S;
  return rows > ROWS && S == 1 ? 0 : svdq::align256(size_t(S) * size_t(rows) * size_t(N) * 4);
}

// A call's rows [m0, m0 + M); the epilogue's row numbers start at m0 with `e`
struct Call {
  const uint16_t* X;
  int64_t M, K, N;
  svdq::AwqWeight w;
  svdq_act act;
  ResEpilogue e;
  hipStream_t s;
};

template <template <int> class Kernel>
auto by_act(svdq_act a) {
  return a == SVDQ_SILU ? Kernel<SVDQ_SILU>::get()
         : a == SVDQ_GELU ? Kernel<SVDQ_GELU>::get()
                          : Kernel<SVDQ_NO_ACT>::get();
}
template <int ACT>
struct SumKernel {
  static auto get() { return res_sum_kernel<ACT>; }
};
template <int ACT>
struct MidKernel {
  static auto get() { return res_mid_kernel<ACT>; }
};
template <int ACT>
struct TwinKernel {
  static auto get() { return res_twin_kernel<ACT>; }
};
template <int ACT>
struct SplitKernel {
  static auto get() { return res_split_kernel<ACT>; }
};
template <int ACT>
struct JoinKernel {
  static auto get() { return res_join_kernel<ACT>; }
};
template <int ACT>
struct WideKernel {
  static auto get() { return res_wide_kernel<ACT>; }
};

svdq_status sum(const Call& c, const float* part, int S) {
  hipLaunchKernelGGL(by_act<SumKernel>(c.act), dim3(unsigned((c.M * c.N / 4 + 63) / 64)), dim3(64),
                     0, c.s, part, S, int(c.M), int(c.N), c.e);
  return svdq::check_launch("awq_res (sum)");
}

template <int MT>
svdq_status few(const Call& c, float* part) {
  if (one_launch(c.M, c.K, c.N)) {
    auto k = c.act == SVDQ_SILU   ? res_column_kernel<MT, SVDQ_SILU>
             : c.act == SVDQ_GELU ? res_column_kernel<MT, SVDQ_GELU>
                                  : res_column_kernel<MT, SVDQ_NO_ACT>;
    hipLaunchKernelGGL(k, dim3(unsigned(c.N / 16)), dim3(NT), 0, c.s, c.X, int(c.M), int(c.K),
                       int(c.N), c.w, c.e);
    return svdq::check_launch("awq_res (column)");
  }
  const Split p = split(c.M, c.K, c.N);
  // chunks of X that fit LDS, a multiple of the register ring's 4: chunk c of a piece is
  // in slot c % 4, which goes on over the pieces
  const int most = int((LDS_X / c.M - 16) / 128 / 4 * 4);
  const int len = int((c.K / 64 + p.slices - 1) / p.slices);
  const int sub = std::min(most, (len + 3) / 4 * 4);
  hipLaunchKernelGGL(res_slice_kernel<MT>, dim3(unsigned(p.blocks * p.slices)), dim3(NT),
                     size_t(c.M) * (sub * 128 + 16), c.s, c.X, int(c.M), int(c.K), int(c.N), c.w,
                     p.slices, sub, part);
  SVDQ_TRY(svdq::check_launch("awq_res (slice)"));
  return sum(c, part, p.slices);
}

svdq_status mid(const Call& c, float* part) {
  const int64_t tiles = mid_tiles(c.M, c.N);
  const svdq_plan::Medium f = svdq_plan::medium(c.M, shape_of(c.K, c.N));
  const int S = f.S;
  svdq_mid::Args p{{c.X, c.X}, c.K, int(c.K / 64), 1, int(c.M)};
  auto k = f.twin ? by_act<TwinKernel>(c.act) : by_act<MidKernel>(c.act);
  hipLaunchKernelGGL(k, dim3(unsigned(tiles * S)), dim3(svdq_mid::NT * (f.twin ? 2 : 1)), 0, c.s, p,
                     c.w, int(c.N), S, int(tiles), c.e, part);
  SVDQ_TRY(svdq::check_launch("awq_res (mid)"));
  return S == 1 ? SVDQ_OK : sum(c, part, S);
}

svdq_status wide(const Call& c, uint16_t* B, const svdq_gemm::Rounds& r, float* part) {
  const int64_t along = (c.K / 64 + DEQUANT_GROUPS - 1) / DEQUANT_GROUPS;
  hipLaunchKernelGGL(res_dequant_kernel, dim3(unsigned((c.N + 63) / 64 * along)), dim3(256), 0, c.s,
                     c.w, int(c.K), int(c.N), B);
  SVDQ_TRY(svdq::check_launch("awq_res (dequant)"));
  svdq_gemm::Args p{{c.X, c.X}, c.K, int(c.K / 64), 1, B, int(c.M), int(c.N)};
  if (r.S > 1) {
    hipLaunchKernelGGL(by_act<SplitKernel>(c.act), dim3(unsigned(r.full + r.left * r.S)),
                       dim3(svdq_gemm::NT), 0, c.s, p, c.e, r.full, r.S, part);
    SVDQ_TRY(svdq::check_launch("awq_res (split)"));
    hipLaunchKernelGGL(by_act<JoinKernel>(c.act), dim3(unsigned(r.left * 32)), dim3(256), 0, c.s, part,
                       r.S, r.full, int(c.M), int(c.N), c.e);
    return svdq::check_launch("awq_res (join)");
  }
  const int64_t tiles = (c.M + 255) / 256 * ((c.N + 255) / 256);
  hipLaunchKernelGGL(by_act<WideKernel>(c.act), dim3(unsigned(tiles)), dim3(svdq_gemm::NT), 0, c.s,
                     p, c.e);
  return svdq::check_launch("awq_res (wide)");
}

// ------------------------------------------------------------- backward
// A wave takes 512 columns, 8 to a lane, and every fourth pair of rows of a workgroup's;
// the workgroup's sums for dgate meet in LDS and, where an image has more workgroups than
// one, in a second launch in a fixed order.  Memory bound: 4608 rows of 12288, 340 MB, 66
// us, 5.2 TB/s, and 5 for the sums.

constexpr int PAIR = 2;                  // rows whose loads a wave has in flight together

template <int ACT, bool DY16>
__global__ __launch_bounds__(256) void res_grad_kernel(const void* __restrict__ dY,
                                                       const uint16_t* __restrict__ Z,
                                                       svdq::Vec gate, int64_t rows, int parts,
                                                       int N, uint16_t* __restrict__ dZ,
                                                       float* __restrict__ part) {
  __shared__ float red[3][8][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (N + 511) / 512;
  const int64_t n = int64_t(blockIdx.x % blocks) * 512 + 8 * lane;
  const int64_t group = blockIdx.x / blocks, image = group / parts, p = group % parts;
  const int64_t r0 = image * rows + p * rows / parts, r1 = image * rows + (p + 1) * rows / parts;
  const bool live = n < N;
  float g[8], acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = 1.f, acc[i] = 0.f;
  if (gate.p && live) load_any<8>(gate.p, gate.b16, image * gate.ld + n, g);
  if (live)
    for (int64_t m = r0 + PAIR * wave; m < r1; m += 4 * PAIR) {
      // (a row past the last is the last one again, and counts for nothing)
      uint32_t d[PAIR][DY16 ? 4 : 8], z[PAIR][4] = {};
#pragma unroll
      for (int k = 0; k < PAIR; ++k) {
        const int64_t at = min(m + k, r1 - 1) * N + n;
        __builtin_memcpy(d[k], static_cast<const uint8_t*>(dY) + at * (DY16 ? 2 : 4), DY16 ? 16 : 32);
        if (Z) __builtin_memcpy(z[k], Z + at, 16);
      }
#pragma unroll
      for (int k = 0; k < PAIR; ++k) {
        if (m + k >= r1) break;
        uint32_t o[4];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t zw = z[k][i / 2];
          float a = __uint_as_float(i & 1 ? zw & 0xFFFF0000u : zw << 16), da = 1.f;
          float dv;
          if constexpr (DY16) {
            const uint32_t dw = d[k][i / 2];
            dv = __uint_as_float(i & 1 ? dw & 0xFFFF0000u : dw << 16);
          } else {
            dv = __uint_as_float(d[k][i]);
          }
          if constexpr (ACT != SVDQ_NO_ACT) {
            const float x = a;
            gate_act_grad<ACT>(x, a, da);
          }
          acc[i] = fmaf(dv, a, acc[i]);
          v[i] = dv * (g[i] * da);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4*>(dZ + (m + k) * N + n) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  if (!part) return;
  if (wave)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave - 1][i][lane] = acc[i];
  __syncthreads();
  if (wave || !live) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    acc[i] = (acc[i] + red[0][i][lane]) + (red[1][i][lane] + red[2][i][lane]);
  float4* const o = reinterpret_cast<float4*>(part + group * N + n);
  o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

template <int ACT>
struct GradKernel {
  static auto get() { return res_grad_kernel<ACT, true>; }
};
template <int ACT>
struct GradKernel32 {
  static auto get() { return res_grad_kernel<ACT, false>; }
};

// Workgroups an image for each 512 columns: about 1024 in all, of 8 to 64 rows
int grad_parts(int64_t M, int64_t N, int64_t images) {
  const int64_t rows = M / images, each = M * ((N + 511) / 512) / 1024;
  return int((rows + std::min<int64_t>(64, std::max<int64_t>(8, each)) - 1) /
             std::min<int64_t>(64, std::max<int64_t>(8, each)));
}

size_t grad_part_bytes(int64_t M, int64_t N, int64_t images) {
  const int64_t groups = images * grad_parts(M, N, images);
  return groups == 1 ? 0 : svdq::align256(size_t(groups) * size_t(N) * 4);
}

}  // namespace

namespace svdq {

size_t awq_res_workspace(int64_t M, int64_t K, int64_t N) {
  svdq_gemm::Rounds r;
  const int64_t w = wide_rows(M, K, N, &r);
  return (w ? weight_bytes(K, N) : 0) + (r.S > 1 ? rounds_bytes(r) : part_bytes(M - w, K, N));
}

svdq_status launch_awq_res(const uint16_t* X, int64_t M, int64_t K, int64_t N, AwqWeight wt,
                           svdq_act act, const ResEpilogue& e, void* ws, hipStream_t s) {
  svdq_gemm::Rounds r;
  const int64_t w = wide_rows(M, K, N, &r), rest = M - w;
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  float* const part = reinterpret_cast<float*>(w8 + (w ? weight_bytes(K, N) : 0));
  Call c{X, M, K, N, wt, act, e, s};
  if (w) {
    c.M = w;
    SVDQ_TRY(wide(c, reinterpret_cast<uint16_t*>(w8), r, part));
  }
  if (!rest) return SVDQ_OK;
  // the rows behind: every operand from row w on; `first` keeps the images' count
  c.X = X + w * K;
  c.M = rest;
  c.e.first = int(w);
  c.e.Y = static_cast<uint8_t*>(e.Y) + w * N * (e.y16 ? 2 : 4);
  if (e.R) c.e.R = static_cast<const uint8_t*>(e.R) + w * N * (e.r16 ? 2 : 4);
  if (e.Z) c.e.Z = e.Z + w * N;
  if (rest > ROWS) return mid(c, part);
  switch ((rest + 15) / 16) {
    case 1: return few<1>(c, part);
    case 2: return few<2>(c, part);
    case 3: return few<3>(c, part);
    default: return few<4>(c, part);
  }
}

size_t awq_res_grad_workspace(int64_t M, int64_t K, int64_t N, int64_t images) {
  return grad_part_bytes(M, N, images) + awq_grad_product_workspace(M, K, N);
}

svdq_status launch_awq_res_grad(const void* dY, bool dy16, const uint16_t* Z, int64_t M, int64_t K,
                                int64_t N, int64_t images, AwqWeight wt, svdq_act act, Vec gate,
                                uint16_t* dX, uint16_t* dZ, float* dgate, void* ws, hipStream_t s) {
  const int64_t rows = M / images, each = gate.ld ? images : 1;
  Joins j{};
  j.images = images;
  if (M == 0) {
    if (dgate) j.add(nullptr, dgate, each);
    return launch_joins(j, N, s);
  }
  if (dy16 && !dgate && awq_res_grad_fused(M, K, N))
    return launch_awq_res_grad_rows(static_cast<const uint16_t*>(dY), Z, M, K, N, images, wt, act,
                                    gate, dX, dZ, ws, s);
  const int parts = grad_parts(M, N, images);
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  // one workgroup's sums are the gradient
  const bool direct = images * parts == each;
  float* const part = !dgate ? nullptr : direct ? dgate : reinterpret_cast<float*>(w8);
  auto k = dy16 ? by_act<GradKernel>(act) : by_act<GradKernel32>(act);
  // a launch of at most 2^23 workgroups (a grid has fewer than 2^32 threads): 2^20 images
  // of one row take several from 8 x 512 columns on
  const int64_t blocks = (N + 511) / 512, most = (int64_t(1) << 23) / (blocks * parts);
  const int64_t step = std::max<int64_t>(1, most);
  for (int64_t i = 0; i < images; i += step) {
    const int64_t n = std::min(step, images - i), at = i * rows * N;
    Vec g = gate;
    if (g.p) g.p = static_cast<const uint8_t*>(g.p) + i * g.ld * (g.b16 ? 2 : 4);
    hipLaunchKernelGGL(k, dim3(unsigned(blocks * n * parts)), dim3(256), 0, s,
                       static_cast<const uint8_t*>(dY) + at * (dy16 ? 2 : 4), Z ? Z + at : nullptr, g,
                       rows, parts, int(N), dZ + at, part ? part + i * parts * N : nullptr);
    SVDQ_TRY(check_launch("awq_res_grad"));
  }
  j.parts = parts;
  if (dgate && !direct) j.add(part, dgate, each);
  SVDQ_TRY(launch_joins(j, N, s));
  return launch_awq_grad_product(dZ, M, K, N, wt, dX, w8 + grad_part_bytes(M, N, images), s);
}

}  // namespace svdq
