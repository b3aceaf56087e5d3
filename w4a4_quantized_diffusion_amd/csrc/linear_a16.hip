// SVDQ layer on few rows with unquantized activations (gfx950).
//
//   Xh = fl32(X smooth),  LR = X lora_down^T (fp32)
//   Y  = [ts_w] sum_g s_g sum_{k in g} Xh q + LR lora_up^T + b
//
// The layer's 4-bit weights (INT4 fold codes with an fp32 scale per 64, NVFP4
// codes with an E4M3 scale per 16) against activations in their own
// precision: what a pooled vector, a time step or a decoding batch of a
// quantized model needs, where quantizing the few activations saves nothing.
//
// Measured, both launches: one row 4096 -> 24576 INT4 (59 MB) 15 us, of which the
// first launch takes 11.2 (5.2 TB/s, part of it from the Infinity Cache); 7 rows
// 4096 -> 12288 NVFP4 13.5 us; 61 rows 2752 -> 10928 in three terms 27 us, shared by
// the partial sums (9 us), the terms of Xh (4) and the products (5 for the terms
// beyond the first); 1024 x 1024 one row 6.2 us, two launches and two trips to
// memory.

#include "w4a16.h"

using namespace svdq_dev;

namespace {

// A float as a sum of T bf16 terms, largest first: two terms hold it to 2^-17,
// three to 2^-24 (each term is the rounding of what the ones before left; the
// subtractions are exact).  An infinite value, and one from 0x1.FFp127 on, whose
// rounding overflows, gives an infinity and NaN: their row of Y is NaN.  (Terms that
// keep the infinity cost the 61-row case its registers, 29 to 38 us.)
template <int T>
__device__ __forceinline__ void split_bf16(const float (&x)[8], uint4 (&t)[T]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int n = 0; n < T; ++n) {
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      w[p] = pack_bf16x2(r[2 * p], r[2 * p + 1]);
      if (n + 1 < T) {
        r[2 * p] -= __uint_as_float(w[p] << 16);
        r[2 * p + 1] -= __uint_as_float(w[p] & 0xFFFF0000u);
      }
    }
    t[n] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 8 elements of X in either type: the loads alone, and their values.  (The
// branch holds nothing but loads, so several can be in flight.)
struct Raw8 {
  uint4 a, b;
};

__device__ __forceinline__ Raw8 load_raw8(const void* X, bool xbf16, int64_t at) {
  Raw8 r;
  r.b = make_uint4(0, 0, 0, 0);
  if (xbf16) {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + at);
  } else {
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(X) + at);
    r.a = f[0];
    r.b = f[1];
  }
  return r;
}

__device__ __forceinline__ void values8(const Raw8& w, bool xbf16, float (&v)[8]) {
  const uint32_t u[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = __uint_as_float(!xbf16 ? u[i] : i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
}

__device__ __forceinline__ void load8(const float* f, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(f)[0], b = reinterpret_cast<const float4*>(f)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int D = 2;                     // chunks of weights in flight per wave
// LDS for the terms of Xh; the second where every workgroup has a compute unit to
// itself (the fewer times the terms are made anew: 61 rows 2752 -> 10928 28.7 to 27.4
// us, 64 rows 4096 -> 12288 31.6 to 29.5)
constexpr int LDS_X = 64 << 10, LDS_ALONE = 152 << 10;
constexpr int SUM_SLICES = 8;            // slices of K that the second launch loads at once
constexpr int LR_STEPS = 4;              // steps of 32 k per wave of LR, loaded at once
constexpr int MAX_LR = 4;

// slices of K over which LR is computed: two rounds of loads each (it runs beside
// the weights' stream, and the second launch waits for every slice's sum)
int lr_slices(int64_t K) {
  constexpr int64_t steps = 2 * WAVES * LR_STEPS;
  return int(std::min<int64_t>(MAX_LR, (K / 32 + steps - 1) / steps));
}

// Lane group j of a wave holds 8 bytes of a weight row's chunk: for INT4 the
// fold format's chunk j (k = 8j + i, then 32 + 8j + i), for NVFP4 block j (k =
// 16j + i, then 16j + 8 + i).  Operand half h of lane group j is at position
// 32h + 8j of the chunk in LDS; this is the k of its first element.
template <int PREC>
__device__ __forceinline__ int operand_k(int h, int j) {
  return PREC == SVDQ_INT4 ? 32 * h + 8 * j : 16 * j + 8 * h;
}

typedef uint32_t v6u __attribute__((ext_vector_type(6)));
typedef __bf16 v32bf __attribute__((ext_vector_type(32)));

// 16 INT4 codes in the fold format: the three words of their 6-bit fields
__device__ __forceinline__ void unfold(uint2 w, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = w.x & ~0x18618618u;
  b = (w.x & 0x18618618u) | (w.y & 0x61861861u);
  c = w.y & ~0x61861861u;
}

// One column's 16 weights of a chunk as two matrix operands.
// INT4: the codes, exact in bf16 (the scale follows the product).  A field
// is the FP6-E2M3 subnormal q / 8, so the conversion with scale 8 gives q.
// NVFP4: e2m1 * e4m3, at most 6 significant bits, exact in bf16.
template <int PREC, int CT>
__device__ __forceinline__ void decode(const uint2 (&w)[CT], const uint32_t (&sc)[CT], int j,
                                       v8bf (&b)[CT][2]) {
  if constexpr (PREC == SVDQ_INT4) {
#pragma unroll
    for (int t = 0; t < CT; t += 2) {
      uint32_t o[6];
      unfold(w[t], o[0], o[1], o[2]);
      unfold(w[t + 1 < CT ? t + 1 : t], o[3], o[4], o[5]);
      const v32bf v = __builtin_amdgcn_cvt_scalef32_pk32_bf16_fp6(
          v6u{o[0], o[1], o[2], o[3], o[4], o[5]}, 8.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[t][0][i] = v[i];
        b[t][1][i] = v[8 + i];
        if (t + 1 < CT) {
          b[t + 1][0][i] = v[16 + i];
          b[t + 1][1][i] = v[24 + i];
        }
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      // E4M3 byte j of the row's four (never negative): its bits shifted by 20
      // are the fp32 bits of v 2^-120
      const float s = __uint_as_float(((sc[t] >> (8 * j)) & 0x7Fu) << 20) * 0x1p120f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = h ? w[t].y : w[t].x;
        const v2f32_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
        const v2f32_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
        const v2f32_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
        const v2f32_t v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
        b[t][h] = __builtin_bit_cast(
            v8bf, make_uint4(pack_bf16x2(v0.x * s, v0.y * s), pack_bf16x2(v1.x * s, v1.y * s),
                             pack_bf16x2(v2.x * s, v2.y * s), pack_bf16x2(v3.x * s, v3.y * s)));
      }
    }
  }
}

// Partial sums of LR = X lora_down^T: a 16 x 16 block over one of LS slices of
// K, [LS][M][rank]; the waves split the slice.
__device__ __forceinline__ void lr_block(int block, const void* __restrict__ X, bool xbf16, int M,
                                         int K, int rank, int LS,
                                         const uint16_t* __restrict__ down,
                                         float* __restrict__ LR, v4f* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane >> 4, r = lane & 15;
  const int rt = rank / 16, sl = block % LS, tile = block / LS;
  const int m0 = tile / rt * 16, i0 = tile % rt * 16;
  const int m = min(m0 + r, M - 1), steps = K / 32;
  v4f acc = {0, 0, 0, 0};
  for (int s0 = sl * WAVES + wave; s0 < steps; s0 += LR_STEPS * WAVES * LS) {
    Raw8 x[LR_STEPS];
    uint4 b[LR_STEPS];
#pragma unroll
    for (int q = 0; q < LR_STEPS; ++q) {
      const int64_t k = 32 * int64_t(min(s0 + q * WAVES * LS, steps - 1)) + 8 * j;
      x[q] = load_raw8(X, xbf16, int64_t(m) * K + k);
      b[q] = *reinterpret_cast<const uint4*>(down + int64_t(i0 + r) * K + k);
    }
#pragma unroll
    for (int q = 0; q < LR_STEPS; ++q) {
      if (s0 + q * WAVES * LS >= steps) b[q] = make_uint4(0, 0, 0, 0);
      float v[8];
      values8(x[q], xbf16, v);
      uint4 t[3];
      split_bf16<3>(v, t);
#pragma unroll
      for (int n = 2; n >= 0; --n)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, t[n]),
                                                      __builtin_bit_cast(v8bf, b[q]), acc, 0, 0, 0);
    }
  }
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) acc += red[w * 64 + lane];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (m0 + 4 * j + e < M) LR[(int64_t(sl) * M + m0 + 4 * j + e) * rank + i0 + r] = acc[e];
}

// First launch.  The first `lr_blocks` workgroups compute LR; it is not needed
// before the second launch and costs the others nothing.  Each of the others: 8
// waves of 16 CT columns each, all rows, and the chunks [s G / S, (s + 1) G / S)
// of K.  The terms of Xh for (part of) that slice are computed into LDS once
// and serve all waves; every wave streams its own columns' weights through
// registers, D chunks ahead.  Partial sums go to part [S][M][N].
template <int PREC, int MT, int T, int CT>
__global__ __launch_bounds__(NT, 4) void a16_slice_kernel(
    const void* __restrict__ X, bool xbf16, int M, int K, int N, int rank, int LS, int lr_blocks,
    int S, int sub, const float* __restrict__ smooth, const uint16_t* __restrict__ down,
    const uint8_t* __restrict__ codes, const uint32_t* __restrict__ scales,
    float* __restrict__ LR, float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t lds[];
  if (int(blockIdx.x) < lr_blocks) {
    lr_block(blockIdx.x, X, xbf16, M, K, rank, LS, down, LR, reinterpret_cast<v4f*>(lds));
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane >> 4, r = lane & 15;
  const int G = K / 64;
  const int slice = (blockIdx.x - lr_blocks) % S;
  const int g0 = int(int64_t(slice) * G / S), count = int(int64_t(slice + 1) * G / S) - g0;
  const int64_t n0 = (int64_t((blockIdx.x - lr_blocks) / S) * WAVES + wave) * (16 * CT);

  int64_t ncl[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) ncl[t] = min(n0 + 16 * t + r, int64_t(N) - 1);
  struct Slot {
    uint2 w[CT];
    uint32_t s[CT];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's
  // data), so that the number of loads in flight is fixed
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int64_t row = int64_t(g0 + min(i, count - 1)) * N;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      sl.w[t] = *reinterpret_cast<const uint2*>(codes + (row + ncl[t]) * 32 + 8 * j);
      sl.s[t] = scales[row + ncl[t]];
    }
  };
  v4f acc[MT][CT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < CT; ++t) acc[mt][t] = v4f{0, 0, 0, 0};

  // `sub` chunks (a multiple of D) of Xh at a time in LDS: [T][M] rows of
  // `sub` chunks and 16 bytes, so that 16 rows start in 16 different groups of
  // 4 banks
  const int rowb = sub * 128 + 16;
  int xoff[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xoff[mt] = min(16 * mt + r, M - 1) * rowb + 16 * j;
  for (int c0 = 0; c0 < count; c0 += sub) {
    const int here = min(sub, count - c0);
    if (c0) __syncthreads();
    for (int i = tid; i < M * here * 8; i += NT) {
      const int m = i / (here * 8), o = i - m * (here * 8);
      const int64_t k = 64 * int64_t(g0 + c0 + (o >> 3)) + operand_k<PREC>((o >> 2) & 1, o & 3);
      const Raw8 raw = load_raw8(X, xbf16, int64_t(m) * K + k);
      float x[8], f[8];
      load8(smooth + k, f);
      values8(raw, xbf16, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f[e];
      uint4 t[T];
      split_bf16<T>(x, t);
#pragma unroll
      for (int n = 0; n < T; ++n)
        *reinterpret_cast<uint4*>(lds + (n * M + m) * rowb + 16 * o) = t[n];
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
#pragma unroll
        for (int t = 0; t < CT; ++t) sl.s[t] = live ? sl.s[t] : 0u;
        v8bf b[CT][2];
        decode<PREC, CT>(sl.w, sl.s, j, b);
        const uint8_t* const xc = lds + 128 * min(c + d, here - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          v8bf a[T][2];
#pragma unroll
          for (int n = 0; n < T; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              a[n][h] = *reinterpret_cast<const v8bf*>(xc + xoff[mt] + n * M * rowb + 64 * h);
#pragma unroll
          for (int t = 0; t < CT; ++t) {
            v4f p = PREC == SVDQ_INT4 ? v4f{0, 0, 0, 0} : acc[mt][t];
#pragma unroll
            for (int n = T - 1; n >= 0; --n)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[n][h], b[t][h], p, 0, 0, 0);
            if constexpr (PREC == SVDQ_INT4) {
              const float f = __uint_as_float(sl.s[t]);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[mt][t][e] = fmaf(f, p[e], acc[mt][t][e]);
            } else {
              acc[mt][t] = p;
            }
          }
        }
        fetch(c0 + c + d + D, sl);
      }
  }

#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int64_t n = n0 + 16 * t + r;
    if (n >= N) continue;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = 16 * mt + 4 * j + e;
        // (read by the next launch, on any XCD: past this one's L2 at once)
        if (m < M)
          __builtin_nontemporal_store(acc[mt][t][e], part + (int64_t(slice) * M + m) * N + n);
      }
  }
}

// Second launch: Y = [ts_w] (the slices' sums in order) + LR lora_up^T + bias,
// a block of 16 rows and 16 columns per wave.
template <int T>
__global__ __launch_bounds__(256) void a16_sum_kernel(
    const float* __restrict__ part, int S, const float* __restrict__ LR, int LS, int M, int N,
    int rank, const uint16_t* __restrict__ up, const float* __restrict__ ts_w,
    const void* __restrict__ bias, bool bbf16, void* __restrict__ Y, bool ybf16) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane >> 4, r = lane & 15;
  const int64_t n0 = (int64_t(blockIdx.x) * 4 + wave) * 16, n = n0 + r;
  if (n0 >= N) return;
  const int m0 = 16 * blockIdx.y, ml = min(m0 + r, M - 1);
  // rows past M repeat the last one and are not stored
  const float* p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = part + int64_t(min(m0 + 4 * j + e, M - 1)) * N + n;
  // LR and lora_up for 64 rank indices: halves q of 32
  uint4 u[2];
  float l[2][MAX_LR][8];
  auto load_low = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = i0 + 32 * q + 8 * j;
      u[q] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int s = 0; s < MAX_LR; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) l[q][s][e] = 0.f;
      if (i < rank) {
        u[q] = *reinterpret_cast<const uint4*>(up + n * rank + i);
#pragma unroll
        for (int s = 0; s < MAX_LR; ++s)
          if (s < LS) load8(LR + (int64_t(s) * M + ml) * rank + i, l[q][s]);
      }
    }
  };
  // all loads first; a slice past the last counts as zeros
  if (rank) load_low(0);
  float v[SUM_SLICES][4];
#pragma unroll
  for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[q][e] = p[e][int64_t(min(q, S - 1)) * M * N];
  const float ts = ts_w ? ts_w[0] : 1.f;
  const float bv = !bias   ? 0.f
                   : bbf16 ? bf16_to_f32(static_cast<const uint16_t*>(bias)[n])
                           : static_cast<const float*>(bias)[n];
  __builtin_amdgcn_sched_barrier(0);
  v4f sum = {0, 0, 0, 0}, low = {0, 0, 0, 0};
  for (int i0 = 0; i0 < rank; i0 += 64) {
    if (i0) load_low(i0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int s = 1; s < MAX_LR; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) l[q][0][e] += l[q][s][e];
      uint4 a[T];
      split_bf16<T>(l[q][0], a);
#pragma unroll
      for (int t = T - 1; t >= 0; --t)
        low = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a[t]),
                                                      __builtin_bit_cast(v8bf, u[q]), low, 0, 0, 0);
    }
  }
#pragma unroll
  for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += q < S ? v[q][e] : 0.f;
  for (int q0 = SUM_SLICES; q0 < S; q0 += SUM_SLICES) {
#pragma unroll
    for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[q][e] = p[e][int64_t(min(q0 + q, S - 1)) * M * N];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < SUM_SLICES; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += q0 + q < S ? v[q][e] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t m = m0 + 4 * j + e;
    if (m >= M) continue;
    const float v = sum[e] * ts + low[e] + bv;
    if (ybf16)
      static_cast<uint16_t*>(Y)[m * N + n] = f32_to_bf16(v);
    else
      static_cast<float*>(Y)[m * N + n] = v;
  }
}

// Columns per wave and slices of K: at most 512 workgroups, two to a compute
// unit, so that one streams while the other fills its LDS or stores; of the
// possible numbers the one that leaves the fewest compute units idle (12288
// columns, 7 rows: 5 slices are 240 workgroups and 13.5 us, 6 are 288 and 16.8).
struct Split {
  int ct, blocks, slices;
};

Split split(int64_t M, int64_t K, int64_t N) {
  Split p;
  p.ct = N >= 8192 ? 2 : 1;
  p.blocks = int((N + 16 * WAVES * p.ct - 1) / (16 * WAVES * p.ct));
  const int most = int(std::min<int64_t>({K / 64, SUM_SLICES, std::max(1, 512 / p.blocks)}));
  p.slices = 1;
  double best = 0;
  for (int S = 1; S <= most; ++S) {
    const int64_t n = int64_t(p.blocks) * S;
    const double used = double(n) / double((n + 255) / 256 * 256);
    if (used >= best) best = used, p.slices = S;
  }
  // Narrow layers on more than 16 rows, bound by the products: more slices, of at
  // least 4 chunks, up to 128 workgroups (54 rows 7424 -> 256: 27.4 us in 8 slices,
  // 14.9 in 29; but one row 8.0 and 10.6)
  if (M > 16)
    p.slices = std::max(p.slices, int(std::min<int64_t>({K / 256, 32, 128 / p.blocks})));
  return p;
}

struct Call {
  const void* X;
  bool xbf16;
  int M, K, N, rank;
  const float* smooth;
  const uint16_t *down, *up;
  const uint8_t* codes;
  const uint32_t* scales;
  const float* ts_w;
  const void* bias;
  bool bbf16;
  void* Y;
  bool ybf16;
  float *part, *LR;
  hipStream_t s;
};

template <int PREC, int MT, int T, int CT>
svdq_status run(const Call& c, const Split& p) {
  // chunks of Xh that fit LDS (at least D do: 64 rows x 3 terms x (2 x 128 + 16) = 52 KB)
  const int LS = lr_slices(c.K), lr_blocks = MT * (c.rank / 16) * LS;
  const int room = lr_blocks + p.blocks * p.slices <= 256 ? LDS_ALONE : LDS_X;
  const int most = (room / (c.M * T) - 16) / 128 / D * D;
  const int len = (c.K / 64 + p.slices - 1) / p.slices;
  const int sub = std::min(most, (len + D - 1) / D * D);
  const size_t shm = std::max(size_t(c.M) * T * (sub * 128 + 16), size_t(WAVES) * 1024);
  auto k = a16_slice_kernel<PREC, MT, T, CT>;
  // (the most that any call asks for: the attribute is the function's, and a host
  // thread with a smaller call must not lower it between another's two steps)
  if (shm > (64 << 10))
    SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, LDS_ALONE));
  hipLaunchKernelGGL(k, dim3(unsigned(lr_blocks + p.blocks * p.slices)), dim3(NT), shm, c.s, c.X,
                     c.xbf16, c.M, c.K, c.N, c.rank, LS, lr_blocks, p.slices, sub, c.smooth, c.down,
                     c.codes, c.scales, c.LR, c.part);
  SVDQ_TRY(svdq::check_launch("a16_slice"));
  hipLaunchKernelGGL(a16_sum_kernel<T>, dim3(unsigned((c.N + 63) / 64), MT), dim3(256), 0, c.s,
                     c.part, p.slices, c.LR, LS, c.M, c.N, c.rank, c.up,
                     PREC == SVDQ_NVFP4 ? c.ts_w : nullptr, c.bias, c.bbf16, c.Y, c.ybf16);
  return svdq::check_launch("a16_sum");
}

template <int PREC, int T, int CT>
svdq_status run_rows(const Call& c, const Split& p) {
  switch ((c.M + 15) / 16) {
    case 1: return run<PREC, 1, T, CT>(c, p);
    case 2: return run<PREC, 2, T, CT>(c, p);
    case 3: return run<PREC, 3, T, CT>(c, p);
    default: return run<PREC, 4, T, CT>(c, p);
  }
}

template <int PREC>
svdq_status run_prec(const Call& c, const Split& p) {
  if (c.ybf16) return p.ct == 2 ? run_rows<PREC, 2, 2>(c, p) : run_rows<PREC, 2, 1>(c, p);
  return p.ct == 2 ? run_rows<PREC, 3, 2>(c, p) : run_rows<PREC, 3, 1>(c, p);
}

size_t part_bytes(int64_t M, int64_t K, int64_t N) {
  return svdq::align256(size_t(split(M, K, N).slices) * size_t(M) * size_t(N) * 4);
}

}  // namespace

namespace svdq {

size_t linear_a16_workspace(int64_t M, int64_t K, int64_t N, int rank) {
  return part_bytes(M, K, N) + align256(size_t(lr_slices(K)) * size_t(M) * rank * 4);
}

svdq_status launch_linear_a16(const void* X, svdq_dtype x_dt, int64_t M, int64_t K, int64_t N,
                              int rank, svdq_precision prec, const float* smooth,
                              const uint16_t* down, const uint16_t* up, const uint8_t* wcodes,
                              const void* wscales, const float* ts_w, const void* bias,
                              svdq_dtype bias_dt, void* Y, svdq_dtype y_dt, void* ws,
                              hipStream_t s) {
  const Call c{X, x_dt == SVDQ_BF16, int(M), int(K), int(N), rank, smooth, down, up, wcodes,
               static_cast<const uint32_t*>(wscales), ts_w, bias, bias_dt == SVDQ_BF16, Y,
               y_dt == SVDQ_BF16, static_cast<float*>(ws),
               reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + part_bytes(M, K, N)), s};
  const Split p = split(M, K, N);
  return prec == SVDQ_INT4 ? run_prec<SVDQ_INT4>(c, p) : run_prec<SVDQ_NVFP4>(c, p);
}

}  // namespace svdq
