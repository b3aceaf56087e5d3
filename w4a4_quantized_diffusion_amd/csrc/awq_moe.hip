// A mixture-of-experts layer on AWQ W4A16 experts for few tokens (gfx950):
//
//   e_j, p_j = the top largest of softmax(logits[t]) (ties to the lower expert)
//   Y[t] = sum_j p_j (act(X[t] Wg_e^T) * (X[t] Wu_e^T)) Wd_e^T,   e = e_j
//
// Wg, Wu [E][N, K], Wd [E][K, N] in the AWQ format.  Two launches: the first forms
// H = act(G) * U for every chosen (token, expert) pair, a slot, the second the
// down-projections and their weighted sum.  Both route for themselves: every workgroup
// finds the choices of all tokens in LDS from the logits (at most 64 x 256), about a
// microsecond, where a launch of its own would cost two to three.  The bound is
// reading the chosen experts' weights; slots are sorted by expert, so that each expert's
// weights are read once for all of its tokens.
//
// H enters the second product rounded to bf16 (the MFMAs' type, and what two separate
// layers would hand on); all sums and the weights are fp32, and no atomics touch them:
// results do not depend on the order of workgroups.

#include "block.h"

using namespace svdq_dev;

namespace {

constexpr int MAX_TOKENS = 64, MAX_EXPERTS = 256, MAX_TOP = 16;
constexpr int MAX_SLOTS = MAX_TOKENS * MAX_TOP;

struct Experts {
  svdq::AwqWeight w;
  int64_t stride;         // rows of codes (32 bytes) from expert to expert: K N / 64

  __device__ __forceinline__ svdq::AwqWeight at(int e) const {
    return {w.q + e * stride * 32, w.s + e * stride, w.z + e * stride};
  }
};

struct Moe {
  const uint16_t* X;
  const void* logits;
  bool l16, renorm;
  int T, E, top, K, N;
  Experts gate, up, down;
  uint16_t* H;            // [T top][N]
  uint16_t* Y;
  int32_t* ids;           // [T][top] or NULL
  float* weights;         // [T][top] or NULL
};

// What every workgroup knows of the routing, in LDS
struct Route {
  uint32_t mask[MAX_EXPERTS][2];       // the tokens that chose an expert
  uint16_t first[MAX_EXPERTS];         // an expert's first slot
  uint8_t active[MAX_EXPERTS];         // experts with tokens, in order
  uint8_t token[MAX_SLOTS];            // of a slot
  float weight[MAX_SLOTS];             // of a slot
  uint8_t chosen[MAX_SLOTS];           // [T][top]
  float p[MAX_SLOTS];                  // [T][top]
  int actives;
};

template <int CTRL>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}

// maximum, minimum and sum over 16 neighbouring lanes, in all of them (row rotations by
// 8, 4, 2, 1)
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, ror16<0x128>(v));
  v = max(v, ror16<0x124>(v));
  v = max(v, ror16<0x122>(v));
  return max(v, ror16<0x121>(v));
}
__device__ __forceinline__ uint32_t min16(uint32_t v) {
  v = min(v, ror16<0x128>(v));
  v = min(v, ror16<0x124>(v));
  v = min(v, ror16<0x122>(v));
  return min(v, ror16<0x121>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += __uint_as_float(ror16<0x128>(__float_as_uint(v)));
  v += __uint_as_float(ror16<0x124>(__float_as_uint(v)));
  v += __uint_as_float(ror16<0x122>(__float_as_uint(v)));
  return v + __uint_as_float(ror16<0x121>(__float_as_uint(v)));
}

// A number whose unsigned order is the logits': NaN above all, -0 as 0.  0 is below
// every logit and marks experts that do not exist or are taken.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  if (v != v) return 0xFFFFFFFFu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// All threads of the workgroup.  16 lanes take a token, expert e in lane e % 16.
__device__ __forceinline__ void route(const Moe& a, Route& r) {
  const int tid = threadIdx.x, NT = blockDim.x, l = tid & 15;
  for (int i = tid; i < 2 * MAX_EXPERTS; i += NT) r.mask[i >> 1][i & 1] = 0;
  __syncthreads();
  for (int t = tid >> 4; t < a.T; t += NT >> 4) {
    uint32_t key[MAX_EXPERTS / 16];
    float v[MAX_EXPERTS / 16];
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 16; ++i) {
      const int e = 16 * i + l;
      v[i] = -INFINITY;
      if (16 * i < a.E && e < a.E) {
        const int at = t * a.E + e;
        v[i] = a.l16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at])
                     : static_cast<const float*>(a.logits)[at];
      }
    }
    float top = -INFINITY, sum = 0.f;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 16; ++i) {
      key[i] = 16 * i + l < a.E ? order_key(v[i]) : 0;
      mine = max(mine, key[i]);
    }
    const uint32_t most = max16(mine);
    // (the largest logit again; a NaN stays one)
    top = most == 0xFFFFFFFFu ? NAN : __uint_as_float(most & 0x80000000u ? most ^ 0x80000000u : ~most);
    const bool none = top == -INFINITY;
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 16; ++i)
      if (16 * i < a.E) sum += 16 * i + l < a.E ? expf(v[i] - top) : 0.f;
    sum = sum16(sum);
    float kept = 0.f, first = 0.f;
    for (int j = 0; j < a.top; ++j) {
      uint32_t best = 0, at = 0xFFFFu;
#pragma unroll
      for (int i = 0; i < MAX_EXPERTS / 16; ++i)
        if (16 * i < a.E && key[i] > best) best = key[i], at = 16 * i + l;
      const uint32_t m = max16(best);
      const uint32_t e = min16(best == m ? at : 0xFFFFu);
#pragma unroll
      for (int i = 0; i < MAX_EXPERTS / 16; ++i)
        if (uint32_t(16 * i + l) == e) key[i] = 0;
      // the logit's own bits back from its key
      const float lv = m == 0xFFFFFFFFu ? NAN
                                        : __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m);
      const float x = none ? 0.f : expf(lv - top);
      kept += x;
      // lane j % 16 keeps the j-th choice (top <= 16)
      if (l == j) first = x;
      if (l == 0) {
        r.chosen[t * a.top + j] = uint8_t(e);
        atomicOr(&r.mask[e][t >> 5], 1u << (t & 31));
      }
    }
    if (l < a.top) r.p[t * a.top + l] = none ? 0.f : first / (a.renorm ? kept : sum);
  }
  __syncthreads();
  // slots by expert: first[] and active[] from one wave's running sums
  if (tid < 64) {
    int count[4], c = 0, n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * tid + i;
      count[i] = __popc(r.mask[e][0]) + __popc(r.mask[e][1]);
      c += count[i];
      n += count[i] > 0;
    }
    int sc = c, sn = n;
    for (int d = 1; d < 64; d *= 2) {
      const int pc = __shfl_up(sc, d), pn = __shfl_up(sn, d);
      if (tid >= d) sc += pc, sn += pn;
    }
    if (tid == 63) r.actives = sn;
    sc -= c;
    sn -= n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.first[4 * tid + i] = uint16_t(sc);
      if (count[i]) r.active[sn++] = uint8_t(4 * tid + i);
      sc += count[i];
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * a.top; i += NT) {
    const int t = i / a.top, e = r.chosen[i];
    // tokens below t in the expert's mask
    const uint32_t lo = t < 32 ? (1u << t) - 1 : 0xFFFFFFFFu, hi = t < 32 ? 0 : (1u << (t - 32)) - 1;
    const int s = r.first[e] + __popc(r.mask[e][0] & lo) + __popc(r.mask[e][1] & hi);
    r.token[s] = uint8_t(t);
    r.weight[s] = r.p[i];
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[i] = e;
      if (a.weights) a.weights[i] = r.p[i];
    }
  }
  __syncthreads();
}

// one chunk of 64 k of 16 rows of weights: lane group j holds k = 16 j .. 16 j + 15
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

// ------------------------------------------------------- H = act(G) * U
// A workgroup's 8 waves own 16 columns of an expert's gate and up projections, take the
// chunks of K in turn, and their sums meet in LDS.

constexpr int UP_WAVES = 8;

// slots s0 .. s0 + count - 1 (count <= 16 MT) of expert e, columns 16 block ..
template <int MT, int ACT>
__device__ __forceinline__ void up_tile(const Moe& a, const Route& r, v4f (*red)[64], int e,
                                        int block, int s0, int count) {
  constexpr int D = MT == 1 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane >> 4, c16 = lane & 15;
  const int64_t n = int64_t(block) * 16 + c16;
  const int G = a.K / 64, chunks = (G - wave + UP_WAVES - 1) / UP_WAVES;
  const svdq::AwqWeight wg = a.gate.at(e), wu = a.up.at(e);
  const uint16_t* xrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    xrow[mt] = a.X + int64_t(r.token[s0 + min(16 * mt + c16, count - 1)]) * a.K + 16 * j;
  struct Slot {
    Codes c[2];
    uint4 x[MT][2];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's data; a wave
  // without chunks loads chunk 0 and never uses it)
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int c = chunks > 0 ? wave + UP_WAVES * min(i, chunks - 1) : 0;
    const int64_t at = int64_t(c) * a.N + n;
    fetch_codes(sl.c[0], wg, at, j);
    fetch_codes(sl.c[1], wu, at, j);
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
  for (int c = 0; c < chunks; c += D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Slot& sl = ring[d];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8bf b[2];
        operands(sl.c[t], c + d < chunks, b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(v8bf, sl.x[mt][h]), b[h], acc[mt][t], 0, 0, 0);
      }
      fetch(c + d + D, sl);
    }
  __syncthreads();                       // the sums of the tile before have been read
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < 2; ++t) red[(wave * MT + mt) * 2 + t][lane] = acc[mt][t];
  __syncthreads();
  if (wave >= MT) return;
  v4f v[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    v[t] = red[2 * wave + t][lane];
#pragma unroll
    for (int w = 1; w < UP_WAVES; ++w) v[t] += red[(w * MT + wave) * 2 + t][lane];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = 16 * wave + 4 * j + i;
    if (s < count)
      a.H[int64_t(s0 + s) * a.N + n] = f32_to_bf16(gate_act<ACT>(v[0][i]) * v[1][i]);
  }
}

template <int ACT>
__global__ __launch_bounds__(64 * UP_WAVES, 4) void moe_up_kernel(Moe a) {
  __shared__ Route r;
  __shared__ v4f red[UP_WAVES * 4 * 2][64];
  route(a, r);
  const int blocks = a.N / 16, items = r.actives * blocks;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int e = r.active[i / blocks], block = i % blocks;
    const int count = __popc(r.mask[e][0]) + __popc(r.mask[e][1]), s0 = r.first[e];
    if (count <= 16)
      up_tile<1, ACT>(a, r, red, e, block, s0, count);
    else if (count <= 32)
      up_tile<2, ACT>(a, r, red, e, block, s0, count);
    else
      up_tile<4, ACT>(a, r, red, e, block, s0, count);
  }
}

// ---------------------------------------------------- the down-projections
// A workgroup owns 16 columns of Y.  Its 16 waves take the active experts in turn (in
// parts of the reduction where the experts are few), add each expert's rows to the
// tokens' sums, a set of them per wave in LDS, and the sets are joined in order.

constexpr int DOWN_WAVES = 16;

template <int MT>
__device__ __forceinline__ void down_tile(const Moe& a, const Route& r, float* out, int e, int64_t n,
                                          int c0, int c1, int s0, int count) {
  constexpr int D = MT == 4 ? 2 : 4;
  const int lane = threadIdx.x & 63, j = lane >> 4, c16 = lane & 15;
  const svdq::AwqWeight w = a.down.at(e);
  const uint16_t* hrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    hrow[mt] = a.H + int64_t(s0 + min(16 * mt + c16, count - 1)) * a.N + 16 * j;
  struct Slot {
    Codes c;
    uint4 x[MT][2];
  } ring[D];
  auto fetch = [&](int i, Slot& sl) __attribute__((always_inline)) {
    const int c = min(i, c1 - 1);
    fetch_codes(sl.c, w, int64_t(c) * a.K + n, j);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4* const x = reinterpret_cast<const uint4*>(hrow[mt] + 64 * int64_t(c));
      sl.x[mt][0] = x[0];
      sl.x[mt][1] = x[1];
    }
  };
  v4f acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) acc[mt] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(c0 + d, ring[d]);
  for (int c = c0; c < c1; c += D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      v8bf b[2];
      operands(ring[d].c, c + d < c1, b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, ring[d].x[mt][h]), b[h], acc[mt], 0, 0, 0);
      fetch(c + d + D, ring[d]);
    }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = 16 * mt + 4 * j + i;
      if (s < count) {
        float* const o = out + r.token[s0 + s] * 16 + c16;
        *o = fmaf(r.weight[s0 + s], acc[mt][i], *o);
      }
    }
}

__global__ __launch_bounds__(64 * DOWN_WAVES) void moe_down_kernel(Moe a) {
  __shared__ Route r;
  extern __shared__ __align__(16) float sums[];     // [wave][T][16]
  route(a, r);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* const out = sums + wave * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 64) out[i] = 0.f;
  const int64_t n = int64_t(blockIdx.x) * 16 + (lane & 15);
  const int G = a.N / 64, actives = r.actives;
  const int parts = min(G, (DOWN_WAVES + actives - 1) / actives);
  for (int u = wave; u < actives * parts; u += DOWN_WAVES) {
    const int e = r.active[u / parts], p = u % parts;
    const int c0 = p * G / parts, c1 = (p + 1) * G / parts;
    const int count = __popc(r.mask[e][0]) + __popc(r.mask[e][1]), s0 = r.first[e];
    if (count <= 16)
      down_tile<1>(a, r, out, e, n, c0, c1, s0, count);
    else if (count <= 32)
      down_tile<2>(a, r, out, e, n, c0, c1, s0, count);
    else
      down_tile<4>(a, r, out, e, n, c0, c1, s0, count);
  }
  __syncthreads();
  if (tid >= a.T * 16) return;
  float v = 0.f;
  for (int w = 0; w < DOWN_WAVES; ++w) v += sums[w * a.T * 16 + tid];
  a.Y[int64_t(tid >> 4) * a.K + int64_t(blockIdx.x) * 16 + (tid & 15)] = f32_to_bf16(v);
}

}  // namespace

namespace svdq {

size_t awq_moe_workspace(int64_t T, int64_t top, int64_t N) { return align256(size_t(T * top * N * 2)); }

svdq_status launch_awq_moe(const uint16_t* X, const void* logits, bool l16, int64_t T, int64_t E,
                           int64_t top, int64_t K, int64_t N, AwqWeight gate, AwqWeight up,
                           AwqWeight down, svdq_act act, bool renorm, uint16_t* Y, int32_t* ids,
                           float* weights, void* ws, hipStream_t s) {
  const int64_t rows = K * N / 64;
  const Moe a{X, logits, l16, renorm, int(T), int(E), int(top), int(K), int(N),
              {gate, rows}, {up, rows}, {down, rows}, static_cast<uint16_t*>(ws), Y, ids, weights};
  const int64_t items = std::min(E, T * top) * (N / 16);
  auto k = act == SVDQ_SILU ? moe_up_kernel<SVDQ_SILU> : moe_up_kernel<SVDQ_GELU>;
  hipLaunchKernelGGL(k, dim3(unsigned(std::min<int64_t>(items, 512))), dim3(64 * UP_WAVES), 0, s, a);
  SVDQ_TRY(check_launch("awq_moe (up)"));
  const size_t lds = size_t(DOWN_WAVES) * size_t(T) * 16 * 4;
  // (the most that any call asks for: the attribute is the function's, and a host
  // thread with fewer tokens must not lower it between another's two steps)
  SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(moe_down_kernel),
                                     hipFuncAttributeMaxDynamicSharedMemorySize,
                                     DOWN_WAVES * MAX_TOKENS * 16 * 4));
  hipLaunchKernelGGL(moe_down_kernel, dim3(unsigned(K / 16)), dim3(64 * DOWN_WAVES), lds, s, a);
  return check_launch("awq_moe (down)");
}

}  // namespace svdq
