// Gated feed-forward pair of AWQ W4A16 layers (gfx950), in one kernel:
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

// 64 rows x 64 columns of both products per workgroup, 4 waves of 32 x 32;
// 64 reduction values at a time are staged (weights dequantized) in LDS.
constexpr int TB = 64;
constexpr int ROWB = 144;                // 64 bf16 (128 bytes) + 16 pad

template <int ACT>
__global__ __launch_bounds__(256) void gated_tile_kernel(
    const uint16_t* __restrict__ X, int M, int K, int N, svdq::AwqWeight wg, svdq::AwqWeight wu,
    const uint16_t* __restrict__ bg, const uint16_t* __restrict__ bu, void* __restrict__ H,
    bool hbf16, uint16_t* __restrict__ Gs, uint16_t* __restrict__ Us) {
  __shared__ __align__(16) uint8_t lds[3][TB * ROWB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m0 = int64_t(blockIdx.y) * TB, n0 = int64_t(blockIdx.x) * TB;
  const int row = tid >> 2, piece = tid & 3;
  const int64_t mr = m0 + row < M ? m0 + row : M - 1;
  const int64_t nr = n0 + row < N ? n0 + row : N - 1;
  v16f ag, au;
#pragma unroll
  for (int e = 0; e < 16; ++e) ag[e] = au[e] = 0.f;
  auto stage_w = [&](const svdq::AwqWeight& w, int g, uint8_t* dst) {
    const int64_t at = int64_t(g) * N + nr;
    const uint2 c = *reinterpret_cast<const uint2*>(w.q + at * 32 + piece * 8);
    const float s = bf16_to_f32(w.s[at]), zs = -bf16_to_f32(w.z[at]) * s;
    uint4* d = reinterpret_cast<uint4*>(dst + row * ROWB + piece * 32);
    d[0] = dequant8(c.x, s, zs);
    d[1] = dequant8(c.y, s, zs);
  };
  const int ra = (wave >> 1) * 32 + (lane & 31), rb = (wave & 1) * 32 + (lane & 31);
  for (int g = 0; g < K / 64; ++g) {
    const uint4* xp = reinterpret_cast<const uint4*>(X + mr * K + 64 * g + 16 * piece);
    uint4* d = reinterpret_cast<uint4*>(lds[0] + row * ROWB + piece * 32);
    d[0] = xp[0];
    d[1] = xp[1];
    stage_w(wg, g, lds[1]);
    stage_w(wu, g, lds[2]);
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int o = ks * 32 + (lane >> 5) * 16;
      const v8bf a = *reinterpret_cast<const v8bf*>(lds[0] + ra * ROWB + o);
      const v8bf b = *reinterpret_cast<const v8bf*>(lds[1] + rb * ROWB + o);
      const v8bf c = *reinterpret_cast<const v8bf*>(lds[2] + rb * ROWB + o);
      ag = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, ag, 0, 0, 0);
      au = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, c, au, 0, 0, 0);
    }
    __syncthreads();
  }
  const int64_t n = n0 + rb;
  if (n >= N) return;
  const float vg = bg ? bf16_to_f32(bg[n]) : 0.f, vu = bu ? bf16_to_f32(bu[n]) : 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t m = m0 + (wave >> 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
    if (m >= M) continue;
    const float G = ag[e] + vg, U = au[e] + vu;
    const float h = gate_act<ACT>(G) * U;
    if (hbf16)
      static_cast<uint16_t*>(H)[m * N + n] = f32_to_bf16(h);
    else
      static_cast<float*>(H)[m * N + n] = h;
    if (Gs) {
      Gs[m * N + n] = f32_to_bf16(G);
      Us[m * N + n] = f32_to_bf16(U);
    }
  }
}

// ---------------------------------------------------------- many rows
// The weights are dequantized once into the workspace, 32 rows of Wg and the
// 32 rows of Wu with the same n alternating, so that one wave's two column
// blocks of the product are the G and the U of the same outputs.

// 64 rows of the pair matrix and one group of 64 k per workgroup; rows past N
// are zeros
__global__ __launch_bounds__(256) void pair_dequant_kernel(svdq::AwqWeight wg, svdq::AwqWeight wu,
                                                           int K, int N,
                                                           uint16_t* __restrict__ B) {
  const int row = threadIdx.x >> 2, piece = threadIdx.x & 3;
  const int g = blockIdx.y;
  const int64_t n = int64_t(blockIdx.x) * 32 + (row & 31);
  const svdq::AwqWeight w = row >= 32 ? wu : wg;
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (n < N) {
    const int64_t at = int64_t(g) * N + n;
    const uint2 c = *reinterpret_cast<const uint2*>(w.q + at * 32 + piece * 8);
    const float s = bf16_to_f32(w.s[at]), zs = -bf16_to_f32(w.z[at]) * s;
    a = dequant8(c.x, s, zs);
    b = dequant8(c.y, s, zs);
  }
  uint4* d = reinterpret_cast<uint4*>(B + (int64_t(blockIdx.x) * 64 + row) * K + 64 * g + 16 * piece);
  d[0] = a;
  d[1] = b;
}

template <int ACT>
__global__ __launch_bounds__(svdq_gemm::NT) void gated_wide_kernel(
    svdq_gemm::Args p, int N, const uint16_t* __restrict__ bg, const uint16_t* __restrict__ bu,
    void* __restrict__ H, bool hbf16, uint16_t* __restrict__ Gs, uint16_t* __restrict__ Us) {
  using namespace svdq_gemm;
  __shared__ Stage st0, st1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  int64_t m0, b0;
  tile_origin((p.M + BM - 1) / BM, (p.rows + BN - 1) / BN, BM, BN, m0, b0);
  v16f acc[RBL][CBL];
  zero_acc(acc);
  tile_product(p, m0, b0, st0, st1, acc);

  const int64_t row0 = m0 + wm * WM, col0 = b0 / 2 + wn * 32;
  const int64_t n = col0 + (lane & 31);
  const float vg = bg && n < N ? bf16_to_f32(bg[n]) : 0.f;
  const float vu = bu && n < N ? bf16_to_f32(bu[n]) : 0.f;
  float* const eb = reinterpret_cast<float*>(&st0) + wave * (32 * 36);
  const float none[1] = {0.f};
  v16f o[RBL][1];
  auto store = [&](void* Y, bool b16) {
    if (b16)
      store_wave_tile<RBL, 1, true>(o, none, eb, lane, row0, col0, p.M, N, Y);
    else
      store_wave_tile<RBL, 1, false>(o, none, eb, lane, row0, col0, p.M, N, Y);
  };
#pragma unroll
  for (int i = 0; i < RBL; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      acc[i][0][e] += vg;
      acc[i][1][e] += vu;
    }
  if (Gs) {
#pragma unroll
    for (int i = 0; i < RBL; ++i) o[i][0] = acc[i][0];
    store(Gs, true);
#pragma unroll
    for (int i = 0; i < RBL; ++i) o[i][0] = acc[i][1];
    store(Us, true);
  }
#pragma unroll
  for (int i = 0; i < RBL; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][0][e] = gate_act<ACT>(acc[i][0][e]) * acc[i][1][e];
  store(H, hbf16);
}

constexpr int64_t WIDE_ROWS = 512;      // rows from which the weights are dequantized up front

int64_t pair_rows(int64_t N) { return (N + 31) / 32 * 64; }

}  // namespace

namespace svdq {

size_t awq_gated_workspace(int64_t M, int64_t K, int64_t N) {
  return M < WIDE_ROWS ? 0 : align256(size_t(pair_rows(N)) * size_t(K) * 2);
}

svdq_status launch_awq_gated(const uint16_t* X, int64_t M, int64_t K, int64_t N, AwqWeight wg,
                             AwqWeight wu, const uint16_t* bg, const uint16_t* bu, svdq_act act,
                             void* H, svdq_dtype h_dt, uint16_t* G, uint16_t* U, void* ws,
                             hipStream_t s) {
  const bool hb = h_dt == SVDQ_BF16;
  if (M >= WIDE_ROWS) {
    uint16_t* const B = static_cast<uint16_t*>(ws);
    hipLaunchKernelGGL(pair_dequant_kernel, dim3(unsigned((N + 31) / 32), unsigned(K / 64)),
                       dim3(256), 0, s, wg, wu, int(K), int(N), B);
    SVDQ_TRY(check_launch("pair_dequant"));
    svdq_gemm::Args p{{X, X}, K, int(K / 64), 1, B, K, int(M), int(pair_rows(N))};
    const int64_t tiles = ((M + 255) / 256) * ((pair_rows(N) + 255) / 256);
    auto k = act == SVDQ_SILU ? gated_wide_kernel<SVDQ_SILU> : gated_wide_kernel<SVDQ_GELU>;
    hipLaunchKernelGGL(k, dim3(unsigned(tiles)), dim3(svdq_gemm::NT), 0, s, p, int(N), bg, bu, H, hb,
                       G, U);
    return check_launch("awq_gated (wide)");
  }
  dim3 grid(unsigned((N + TB - 1) / TB), unsigned((M + TB - 1) / TB));
  auto k = act == SVDQ_SILU ? gated_tile_kernel<SVDQ_SILU> : gated_tile_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, grid, dim3(256), 0, s, X, int(M), int(K), int(N), wg, wu, bg, bu, H, hb,
                     G, U);
  return check_launch("awq_gated");
}

}  // namespace svdq
