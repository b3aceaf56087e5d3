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

#include "w4a16.h"

using namespace svdq_dev;

namespace {

// dG, dU of 8 elements per thread
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

constexpr int TB = 64;
constexpr int ROWB = 144;

// 64 rows x one group of 64 columns of dX per workgroup, 64 n at a time.
__global__ __launch_bounds__(256) void grad_tile_kernel(
    const uint16_t* __restrict__ dA, svdq::AwqWeight wa, const uint16_t* __restrict__ dB,
    svdq::AwqWeight wb, int pairs, int M, int K, int N, void* __restrict__ dX, bool xbf16) {
  __shared__ __align__(16) uint8_t lds[2][TB * ROWB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = blockIdx.x;
  const int64_t m0 = int64_t(blockIdx.y) * TB;
  const int row = tid >> 2, piece = tid & 3;
  const int64_t mr = m0 + row < M ? m0 + row : M - 1;
  const int oct = tid >> 5, byte = tid & 31;
  v16f acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  const int ra = (wave >> 1) * 32 + (lane & 31), rb = (wave & 1) * 32 + (lane & 31);
  for (int p = 0; p < pairs; ++p) {
    const uint16_t* const d = p ? dB : dA;
    const svdq::AwqWeight w = p ? wb : wa;
    for (int64_t n0 = 0; n0 < N; n0 += 64) {
      // rows of the last chunk past N (a multiple of 16) count as zeros on both sides
      uint4 a0 = make_uint4(0, 0, 0, 0), a1 = a0;
      if (n0 + 16 * piece < N) {
        const uint4* ap = reinterpret_cast<const uint4*>(d + mr * N + n0 + 16 * piece);
        a0 = ap[0];
        a1 = ap[1];
      }
      uint4* ad = reinterpret_cast<uint4*>(lds[0] + row * ROWB + piece * 32);
      ad[0] = a0;
      ad[1] = a1;
      float lo[8], hi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + 8 * oct + i;
        lo[i] = hi[i] = 0.f;
        if (n < N) {
          const int64_t at = int64_t(g) * N + n;
          const uint32_t c = w.q[at * 32 + byte];
          const float s = bf16_to_f32(w.s[at]), zs = -bf16_to_f32(w.z[at]) * s;
          lo[i] = fmaf(float(c & 15), s, zs);
          hi[i] = fmaf(float(c >> 4), s, zs);
        }
      }
      *reinterpret_cast<uint4*>(lds[1] + (2 * byte) * ROWB + oct * 16) =
          make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                     pack_bf16x2(lo[4], lo[5]), pack_bf16x2(lo[6], lo[7]));
      *reinterpret_cast<uint4*>(lds[1] + (2 * byte + 1) * ROWB + oct * 16) =
          make_uint4(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]),
                     pack_bf16x2(hi[4], hi[5]), pack_bf16x2(hi[6], hi[7]));
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int o = ks * 32 + (lane >> 5) * 16;
        const v8bf a = *reinterpret_cast<const v8bf*>(lds[0] + ra * ROWB + o);
        const v8bf b = *reinterpret_cast<const v8bf*>(lds[1] + rb * ROWB + o);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
      }
      __syncthreads();
    }
  }
  const int64_t k = int64_t(g) * 64 + rb;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t m = m0 + (wave >> 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
    if (m >= M) continue;
    if (xbf16)
      static_cast<uint16_t*>(dX)[m * K + k] = f32_to_bf16(acc[e]);
    else
      static_cast<float*>(dX)[m * K + k] = acc[e];
  }
}

}  // namespace

namespace svdq {

size_t awq_linear_grad_workspace(int64_t M, int64_t K, int64_t N) { return 0; }
size_t awq_gated_grad_workspace(int64_t M, int64_t K, int64_t N) {
  return 2 * align256(size_t(M) * size_t(N) * 2);
}

svdq_status launch_awq_linear_grad(const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                                   AwqWeight w, void* dX, svdq_dtype x_dt, void* ws,
                                   hipStream_t s) {
  dim3 grid(unsigned(K / 64), unsigned((M + TB - 1) / TB));
  hipLaunchKernelGGL(grad_tile_kernel, grid, dim3(256), 0, s, dY, w, dY, w, 1, int(M), int(K),
                     int(N), dX, x_dt == SVDQ_BF16);
  return check_launch("awq_linear_grad");
}

svdq_status launch_awq_gated_grad(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                  int64_t M, int64_t K, int64_t N, AwqWeight wg, AwqWeight wu,
                                  svdq_act act, uint16_t* dX, uint16_t* dG, uint16_t* dU, void* ws,
                                  hipStream_t s) {
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  if (!dG) dG = reinterpret_cast<uint16_t*>(w8);
  if (!dU) dU = reinterpret_cast<uint16_t*>(w8 + align256(size_t(M) * size_t(N) * 2));
  const int64_t n8 = M * N / 8;
  const unsigned blocks = unsigned(std::min<int64_t>((n8 + 255) / 256, 16384));
  auto k = act == SVDQ_SILU ? gate_grad_kernel<SVDQ_SILU> : gate_grad_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(blocks), dim3(256), 0, s, dH, G, U, n8, dG, dU);
  SVDQ_TRY(check_launch("gate_grad"));
  dim3 grid(unsigned(K / 64), unsigned((M + TB - 1) / TB));
  hipLaunchKernelGGL(grad_tile_kernel, grid, dim3(256), 0, s, dG, wg, dU, wu, 2, int(M), int(K),
                     int(N), static_cast<void*>(dX), true);
  return check_launch("awq_gated_grad");
}

}  // namespace svdq
