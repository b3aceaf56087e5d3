// SVDQ layer on few rows with unquantized activations (gfx950).
//
//   Xh = fl32(X smooth),  LR = X lora_down^T (fp32)
//   Y  = [ts_w] sum_g s_g sum_{k in g} Xh q + LR lora_up^T + b
//
// The layer's 4-bit weights (INT4 fold codes with an fp32 scale per 64, NVFP4
// codes with an E4M3 scale per 16) against activations in their own
// precision: what a pooled vector, a time step or a decoding batch of a
// quantized model needs, where quantizing the few activations saves nothing.

#include "w4a16.h"

using namespace svdq_dev;

namespace {

__device__ __forceinline__ float load_x(const void* X, bool xbf16, int64_t i) {
  return xbf16 ? bf16_to_f32(static_cast<const uint16_t*>(X)[i]) : static_cast<const float*>(X)[i];
}

// one wave per (row m, rank index i)
__global__ __launch_bounds__(64) void a16_lr_kernel(const void* __restrict__ X, bool xbf16, int K,
                                                    int rank, const uint16_t* __restrict__ down,
                                                    float* __restrict__ LR) {
  const int m = blockIdx.x / rank, i = blockIdx.x % rank;
  float s = 0.f;
  for (int k = threadIdx.x; k < K; k += 64)
    s = fmaf(load_x(X, xbf16, int64_t(m) * K + k), bf16_to_f32(down[int64_t(i) * K + k]), s);
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if (threadIdx.x == 0) LR[int64_t(m) * rank + i] = s;
}

// the 64 codes of (group, row) as fp32 values
template <int PREC>
__device__ __forceinline__ void decode64(const uint8_t* __restrict__ codes,
                                         const void* __restrict__ scales, int64_t at,
                                         float (&v)[64]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(codes + at * 32);
  if constexpr (PREC == SVDQ_INT4) {
    const float s = static_cast<const float*>(scales)[at];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t x = w[2 * c], y = w[2 * c + 1];
      const uint32_t o[3] = {x & ~0x18618618u, (x & 0x18618618u) | (y & 0x61861861u),
                             y & ~0x61861861u};
#pragma unroll
      for (int f = 0; f < 16; ++f) {
        const int b = 6 * f, i = b / 32, r = b % 32;
        uint32_t p = o[i] >> r;
        if (r > 26) p |= o[i + 1] << (32 - r);
        const float a = float(p & 7);
        v[f < 8 ? 8 * c + f : 32 + 8 * c + f - 8] = ((p >> 5) & 1 ? -a : a) * s;
      }
    }
  } else {
    const uint8_t* sb = static_cast<const uint8_t*>(scales) + at * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = e4m3_value(sb[i / 2]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t c = (w[i] >> (4 * j)) & 15, e = (c >> 1) & 3, m = c & 1;
        const float a = e == 0 ? 0.5f * float(m) : ldexpf(1.f + 0.5f * float(m), int(e) - 1);
        v[8 * i + j] = (c & 8 ? -a : a) * s;
      }
    }
  }
}

// 16 columns per workgroup, 16 threads per column over the groups of K, one
// tile of 4 rows at a time
template <int PREC>
__global__ __launch_bounds__(256) void a16_simple_kernel(
    const void* __restrict__ X, bool xbf16, int M, int K, int N, int rank,
    const float* __restrict__ smooth, const uint8_t* __restrict__ codes,
    const void* __restrict__ scales, const uint16_t* __restrict__ up,
    const float* __restrict__ ts_w, const float* __restrict__ LR, const void* __restrict__ bias,
    bool bbf16, void* __restrict__ Y, bool ybf16) {
  __shared__ float red[16][16][4];
  const int c = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const int64_t n = int64_t(blockIdx.x) * 16 + c;
  for (int m0 = 0; m0 < M; m0 += 4) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g = sl; g < K / 64; g += 16) {
      float v[64];
      decode64<PREC>(codes, scales, int64_t(g) * N + n, v);
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + i < M ? m0 + i : M - 1;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 64; ++k)
          s = fmaf(load_x(X, xbf16, int64_t(m) * K + 64 * g + k) * smooth[64 * g + k], v[k], s);
        acc[i] += s;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[sl][c][i] = acc[i];
    __syncthreads();
    if (sl < 4 && m0 + sl < M) {
      const int m = m0 + sl;
      float s = 0.f;
      for (int t = 0; t < 16; ++t) s += red[t][c][sl];
      if (PREC == SVDQ_NVFP4) s *= ts_w[0];
      for (int i = 0; i < rank; ++i)
        s = fmaf(LR[int64_t(m) * rank + i], bf16_to_f32(up[n * rank + i]), s);
      if (bias)
        s += bbf16 ? bf16_to_f32(static_cast<const uint16_t*>(bias)[n])
                   : static_cast<const float*>(bias)[n];
      if (ybf16)
        static_cast<uint16_t*>(Y)[int64_t(m) * N + n] = f32_to_bf16(s);
      else
        static_cast<float*>(Y)[int64_t(m) * N + n] = s;
    }
    __syncthreads();
  }
}

}  // namespace

namespace svdq {

size_t linear_a16_workspace(int64_t M, int64_t K, int64_t N, int rank) {
  return align256(size_t(M) * rank * 4);
}

svdq_status launch_linear_a16(const void* X, svdq_dtype x_dt, int64_t M, int64_t K, int64_t N,
                              int rank, svdq_precision prec, const float* smooth,
                              const uint16_t* down, const uint16_t* up, const uint8_t* wcodes,
                              const void* wscales, const float* ts_w, const void* bias,
                              svdq_dtype bias_dt, void* Y, svdq_dtype y_dt, void* ws,
                              hipStream_t s) {
  float* LR = static_cast<float*>(ws);
  if (rank) {
    hipLaunchKernelGGL(a16_lr_kernel, dim3(unsigned(M * rank)), dim3(64), 0, s, X,
                       x_dt == SVDQ_BF16, int(K), rank, down, LR);
    SVDQ_TRY(check_launch("a16_lr"));
  }
  auto k = prec == SVDQ_INT4 ? a16_simple_kernel<SVDQ_INT4> : a16_simple_kernel<SVDQ_NVFP4>;
  hipLaunchKernelGGL(k, dim3(unsigned(N / 16)), dim3(256), 0, s, X, x_dt == SVDQ_BF16, int(M),
                     int(K), int(N), rank, smooth, wcodes, wscales, up, ts_w, LR, bias,
                     bias_dt == SVDQ_BF16, Y, y_dt == SVDQ_BF16);
  return check_launch("a16");
}

}  // namespace svdq
