// Shared pieces of the weight-only (W4A16) operators: their entry points behind
// the C ABI, the dequantization of AWQ weights, the gate activations of a gated
// feed-forward block and their derivatives, and the order of output tiles.
#pragma once

#include "internal.h"

#include <algorithm>

#define SVDQ_TRY(x)                       \
  do {                                    \
    svdq_status st_ = (x);                \
    if (st_ != SVDQ_OK) return st_;       \
  } while (0)

namespace svdq {

// an AWQ layer's weights: q [K/64][N][32 bytes], scales and zeros bf16 [K/64][N]
struct AwqWeight {
  const uint8_t* q;
  const uint16_t* s;
  const uint16_t* z;
};
// Bytes of the caller's workspace for valid sizes (a multiple of 256, 0: none)
size_t awq_gated_workspace(int64_t M, int64_t K, int64_t N);
size_t awq_linear_grad_workspace(int64_t M, int64_t K, int64_t N);
size_t awq_gated_grad_workspace(int64_t M, int64_t K, int64_t N);
size_t linear_a16_workspace(int64_t M, int64_t K, int64_t N, int rank);
svdq_status launch_awq_gated(const uint16_t* X, int64_t M, int64_t K, int64_t N, AwqWeight wg,
                             AwqWeight wu, const uint16_t* bg, const uint16_t* bu, svdq_act act,
                             void* H, svdq_dtype h_dt, uint16_t* G, uint16_t* U, void* ws,
                             hipStream_t s);
svdq_status launch_awq_linear_grad(const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                                   AwqWeight w, void* dX, svdq_dtype x_dt, void* ws,
                                   hipStream_t s);
svdq_status launch_awq_gated_grad(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                  int64_t M, int64_t K, int64_t N, AwqWeight wg, AwqWeight wu,
                                  svdq_act act, uint16_t* dX, uint16_t* dG, uint16_t* dU, void* ws,
                                  hipStream_t s);
svdq_status launch_linear_a16(const void* X, svdq_dtype x_dt, int64_t M, int64_t K, int64_t N,
                              int rank, svdq_precision prec, const float* smooth,
                              const uint16_t* down, const uint16_t* up, const uint8_t* wcodes,
                              const void* wscales, const float* ts_w, const void* bias,
                              svdq_dtype bias_dt, void* Y, svdq_dtype y_dt, void* ws,
                              hipStream_t s);

}  // namespace svdq

namespace svdq_dev {

// 8 unsigned nibbles of an AWQ layer (one dword, even k low) -> (q - z) s in k
// order, in fp32 and rounded to bf16 (4 dwords).  zs = -z s (exact in fp32).  A
// byte 0x0q read as FP8-E4M3 is q 2^-9 for every q in 0..15 (a subnormal below 8,
// exponent field 1 from 8 on), so the scaled conversion with the power of two
// 2^9 gives q exactly, two codes per instruction.
__device__ __forceinline__ void dequant8_f32(uint32_t w, float s, float zs, float (&v)[8]) {
  const int e = int(w & 0x0F0F0F0Fu), o = int((w >> 4) & 0x0F0F0F0Fu);
  const v2f32_t q02 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e, 512.0f, false);
  const v2f32_t q46 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e, 512.0f, true);
  const v2f32_t q13 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(o, 512.0f, false);
  const v2f32_t q57 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(o, 512.0f, true);
  v[0] = fmaf(q02.x, s, zs);
  v[1] = fmaf(q13.x, s, zs);
  v[2] = fmaf(q02.y, s, zs);
  v[3] = fmaf(q13.y, s, zs);
  v[4] = fmaf(q46.x, s, zs);
  v[5] = fmaf(q57.x, s, zs);
  v[6] = fmaf(q46.y, s, zs);
  v[7] = fmaf(q57.y, s, zs);
}

__device__ __forceinline__ uint4 dequant8(uint32_t w, float s, float zs) {
  float v[8];
  dequant8_f32(w, s, zs, v);
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

constexpr float LOG2E = 1.44269504088896340736f;

// a = act(x) and d = act'(x), for the SiLU x s, s = 1 / (1 + exp(-x)), and the
// tanh form of GELU, 0.5 x (1 + tanh u) = x s with s = 1 / (1 + exp(-2u)),
// u = sqrt(2/pi) (x + 0.044715 x^3).  With t the sigmoid's argument
// (x or 2u), act' = s + x t' s (1 - s).  exp by exp2 and the reciprocal are
// the hardware's (1 ulp each).  Beyond |x| = 128, s (1 - s) is 0 in fp32 for
// both (s or 1 - s is), and the clamp keeps x t' finite there, so that a large
// |x| gives act' = 0 or 1 and never inf * 0.
template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float x) {
  float t = x;
  if constexpr (ACT == SVDQ_GELU) t = 1.5957691216057308f * (x + 0.044715f * x * x * x);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-t * LOG2E));
}

template <int ACT>
__device__ __forceinline__ float gate_act(float x) {
  return x * gate_sigmoid<ACT>(x);
}

template <int ACT>
__device__ __forceinline__ void gate_act_grad(float x, float& a, float& d) {
  const float s = gate_sigmoid<ACT>(x);
  const float c = fminf(fmaxf(x, -128.f), 128.f);
  float t1 = 1.f;
  if constexpr (ACT == SVDQ_GELU) t1 = 1.5957691216057308f * (1.f + 0.134145f * c * c);
  a = x * s;
  d = s + c * t1 * (s * (1.f - s));
}

// tile_origin for a tile number that is not the workgroup's (blocks of the same
// shape: 8 column tiles wide, a run of them per XCD)
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int bm, int bn,
                                        int64_t& m0, int64_t& n0) {
  constexpr int GN = 8;
  const int total = tiles_m * tiles_n;
  if ((total & 7) == 0) t = (t & 7) * (total >> 3) + (t >> 3);
  const int grp = t / (GN * tiles_m), in = t - grp * (GN * tiles_m);
  const int gn = min(GN, tiles_n - grp * GN);
  m0 = int64_t(in / gn) * bm;
  n0 = int64_t(grp * GN + in % gn) * bn;
}

}  // namespace svdq_dev
