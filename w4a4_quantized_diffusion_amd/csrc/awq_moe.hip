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

__device__ __forceinline__ float key_value(uint32_t key) {
  return key == 0xFFFFFFFFu ? NAN : __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// inclusive sum over a wave's lanes
__device__ __forceinline__ int scan64(int v) {
#define ADD(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xF, true)
  ADD(0x111, 0xF);                       // row_shr 1, 2, 4, 8
  ADD(0x112, 0xF);
  ADD(0x114, 0xF);
  ADD(0x118, 0xF);
  ADD(0x142, 0xA);                       // row_bcast 15, 31
  ADD(0x143, 0xC);
#undef ADD
  return v;
}

// The choices of the tokens, 16 lanes to a token, expert e in lane e % 16; NV values a
// lane (E <= 16 NV).  A lane keeps the token's choice with its number.
template <int NV>
__device__ __forceinline__ void choose(const Moe& a, Route& r) {
  const int tid = threadIdx.x, l = tid & 15;
  for (int t = tid >> 4; t < a.T; t += int(blockDim.x) >> 4) {
    uint32_t key[NV];
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (past the last expert the last one's, and its key is 0)
      const int at = t * a.E + min(16 * i + l, a.E - 1);
      v[i] = a.l16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at])
                   : static_cast<const float*>(a.logits)[at];
    }
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      key[i] = 16 * i + l < a.E ? order_key(v[i]) : 0;
      mine = max(mine, key[i]);
    }
    const float top = key_value(max16(mine));
    const bool none = top == -INFINITY;
    float sum = 0.f, kept = 0.f, p = 0.f;
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += key[i] ? expf(v[i] - top) : 0.f;
      sum = sum16(sum);
    }
    uint32_t choice = 0;
    for (int j = 0; j < a.top; ++j) {
      uint32_t best = 0, at = 0xFFFFu;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] > best) best = key[i], at = 16 * i + l;
      const uint32_t m = max16(best);
      const uint32_t e = min16(best == m ? at : 0xFFFFu);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (uint32_t(16 * i + l) == e) key[i] = 0;
      if (l == j) choice = e, p = expf(key_value(m) - top);
    }
    if (l >= a.top) p = 0.f;
    if (a.renorm) sum = sum16(p);
    p = none ? 0.f : p / sum;
    if (l >= a.top) continue;
    const int i = t * a.top + l;
    r.chosen[i] = uint8_t(choice);
    r.p[i] = p;
    if (a.T == 1) {
      // slots in the order of the choices
      r.mask[choice][0] = 1;
      r.mask[choice][1] = 0;
      r.first[choice] = uint16_t(l);
      r.active[l] = uint8_t(choice);
      r.token[l] = 0;
      r.weight[l] = p;
    } else {
      atomicOr(&r.mask[choice][t >> 5], 1u << (t & 31));
    }
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[i] = int(choice);
      if (a.weights) a.weights[i] = p;
    }
  }
}

// All threads of the workgroup
__device__ __forceinline__ void route(const Moe& a, Route& r) {
  const int tid = threadIdx.x, NT = blockDim.x;
  if (a.T > 1) {
    for (int i = tid; i < 2 * MAX_EXPERTS; i += NT) r.mask[i >> 1][i & 1] = 0;
    __syncthreads();
  } else if (tid == 0) {
    r.actives = a.top;
  }
  if (a.E <= 16)
    choose<1>(a, r);
  else if (a.E <= 32)
    choose<2>(a, r);
  else if (a.E <= 64)
    choose<4>(a, r);
  else if (a.E <= 128)
    choose<8>(a, r);
  else
    choose<16>(a, r);
  __syncthreads();
  if (a.T == 1) return;
  // slots by expert: first[] and active[] from one wave's running sums, 4 experts a lane
  if (tid < 64) {
    int count[4], c = 0, n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * tid + i;
      count[i] = __popc(r.mask[e][0]) + __popc(r.mask[e][1]);
      c += count[i];
      n += count[i] > 0;
    }
    int sc = scan64(c), sn = scan64(n);
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
  }
  __syncthreads();
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int tokens_of(const Route& r, int e) {
  return uniform(__popc(r.mask[e][0]) + __popc(r.mask[e][1]));
}

// 8 codes each of k = 16 j .. 16 j + 7 and 16 j + 8 .. 16 j + 15 of a row's chunk, times
// the row's scale; past the last chunk (not live) the scales are zeros
__device__ __forceinline__ void operands(uint2 w, uint32_t s16, uint32_t z16, bool live,
                                         v8bf (&b)[2]) {
  const float s = live ? __uint_as_float(s16 << 16) : 0.f;
  const float zs = -__uint_as_float(z16 << 16) * s;
  b[0] = __builtin_bit_cast(v8bf, dequant8(w.x, s, zs));
  b[1] = __builtin_bit_cast(v8bf, dequant8(w.y, s, zs));
}

// a barrier for LDS that leaves the loads from memory in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------- H = act(G) * U
// An item is 32 columns of an expert's gate and up projections for 16 MT of its slots.
// A workgroup's 8 waves take the chunks of K in turn, and their sums meet in LDS.  The
// workgroups go on from item to item with the next item's loads in flight.

constexpr int UP_WAVES = 8;

template <int MT>
struct UpCursor {
  int item, e, block, s0, left, step;

  // (the end of the list leaves the cursor where it is; `item` says that it ended)
  __device__ __forceinline__ void open(const Route& r, int blocks, int items) {
    step = 0;
    if (item >= items) return;
    e = uniform(r.active[item / blocks]);
    block = item % blocks;
    s0 = uniform(r.first[e]);
    left = tokens_of(r, e);
  }
};

template <int MT, int ACT>
__global__ __launch_bounds__(64 * UP_WAVES, 4) void moe_up_kernel(Moe a) {
  constexpr int D = MT == 1 ? 3 : 2;
  __shared__ Route r;
  __shared__ float red[UP_WAVES][MT][2][2][4][64];   // [wave][rows][column parity][G, U][e][lane]
  route(a, r);
  const int lane = threadIdx.x & 63, j = lane >> 4, c16 = lane & 15;
  const int wave = uniform(threadIdx.x >> 6);
  const int G = a.K / 64, steps = (G + UP_WAVES - 1) / UP_WAVES;
  const int blocks = a.N / 32, items = uniform(r.actives) * blocks;
  // workgroups are dealt round-robin to the 8 XCDs: each XCD takes a run of items, so that
  // an expert's rows of X and shared lines of scales meet in one L2
  int start = blockIdx.x, stride = gridDim.x, end = items;
  if ((gridDim.x & 7) == 0) {
    const int per = (items + 7) / 8, xcd = blockIdx.x & 7;
    start = xcd * per + (blockIdx.x >> 3);
    end = min(items, (xcd + 1) * per);
    stride = gridDim.x >> 3;
  }
  if (start >= end) return;
  UpCursor<MT> at, ahead;
  at.item = start;
  at.open(r, blocks, end);
  ahead = at;
  auto advance = [&](UpCursor<MT>& c) __attribute__((always_inline)) {
    if (++c.step < steps) return;
    c.step = 0;
    if (c.left > 16 * MT) {
      c.left -= 16 * MT;
      c.s0 += 16 * MT;
      return;
    }
    c.item += stride;
    c.open(r, blocks, end);
  };
  struct Slot {
    uint2 w[2][2];                       // gate, up; column parity
    uint32_t s[2], z[2];                 // of both columns
    uint4 x[MT][2];
  } ring[D];
  const uint16_t* xrow[MT];
  auto rows = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      xrow[mt] = a.X + int64_t(r.token[ahead.s0 + min(16 * mt + c16, ahead.left - 1)]) * a.K + 16 * j;
  };
  rows();
  // every slot is always loaded (past the last chunk with the last one's data), so that
  // the number of loads in flight is fixed
  auto fetch = [&](Slot& sl) __attribute__((always_inline)) {
    const int c = min(wave + UP_WAVES * ahead.step, G - 1);
    const int64_t row = ahead.e * a.gate.stride + int64_t(c) * a.N + 32 * ahead.block;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const svdq::AwqWeight& w = t ? a.up.w : a.gate.w;
      const uint8_t* const q = w.q + row * 32;
#pragma unroll
      for (int p = 0; p < 2; ++p)
        sl.w[t][p] = *reinterpret_cast<const uint2*>(q + uint32_t(64 * c16 + 32 * p + 8 * j));
      sl.s[t] = reinterpret_cast<const uint32_t*>(w.s + row)[c16];
      sl.z[t] = reinterpret_cast<const uint32_t*>(w.z + row)[c16];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4* const x = reinterpret_cast<const uint4*>(xrow[mt] + 64 * int64_t(c));
      sl.x[mt][0] = x[0];
      sl.x[mt][1] = x[1];
    }
    const int s0 = ahead.s0, item = ahead.item;
    advance(ahead);
    if (ahead.s0 != s0 || ahead.item != item) rows();
  };
  v4f acc[MT][2][2];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < 2; ++t) acc[mt][p][t] = v4f{0, 0, 0, 0};
  };
  clear();
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(ring[d]);
  while (true) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Slot& sl = ring[d];
      const bool live = wave + UP_WAVES * at.step < G;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          v8bf b[2];
          operands(sl.w[t][p], p ? sl.s[t] >> 16 : sl.s[t] & 0xFFFF, p ? sl.z[t] >> 16 : sl.z[t] & 0xFFFF,
                   live, b);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[mt][p][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(v8bf, sl.x[mt][h]), b[h], acc[mt][p][t], 0, 0, 0);
        }
      fetch(sl);
      if (at.step == steps - 1) {
        // the waves' sums in order
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) red[wave][mt][p][t][e][lane] = acc[mt][p][t][e];
        clear();
        lds_barrier();
        // wave e of four: rows 4 j + e, both columns
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int e = wave - 4 * (mt & 1), row = 16 * mt + 4 * j + e;
          if (e < 0 || e > 3 || row >= at.left) continue;
          float h[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            float g = red[0][mt][p][0][e][lane], u = red[0][mt][p][1][e][lane];
#pragma unroll
            for (int w = 1; w < UP_WAVES; ++w) {
              g += red[w][mt][p][0][e][lane];
              u += red[w][mt][p][1][e][lane];
            }
            h[p] = gate_act<ACT>(g) * u;
          }
          reinterpret_cast<uint32_t*>(a.H + int64_t(at.s0 + row) * a.N + 32 * at.block)[c16] =
              pack_bf16x2(h[0], h[1]);
        }
        lds_barrier();
      }
      advance(at);
      if (at.item >= end) return;
    }
  }
}

// ---------------------------------------------------- the down-projections
// A workgroup owns 16 columns of Y.  Its 16 waves take the active experts in turn (in
// parts of the reduction where the experts are few), add each expert's rows to the
// tokens' sums, a set of them per wave in LDS, and the sets are joined in order.  A
// wave goes on from expert to expert with the next one's loads in flight.

constexpr int DOWN_WAVES = 16;

template <int MT>
__global__ __launch_bounds__(64 * DOWN_WAVES) void moe_down_kernel(Moe a) {
  constexpr int D = MT == 1 ? 5 : 3;
  __shared__ Route r;
  extern __shared__ __align__(16) float sums[];     // [wave][T][16]
  route(a, r);
  const int tid = threadIdx.x, lane = tid & 63, j = lane >> 4, c16 = lane & 15;
  const int wave = uniform(tid >> 6);
  float* const out = sums + wave * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 64) out[i] = 0.f;
  int cols = blockIdx.x;
  if ((gridDim.x & 7) == 0) cols = (cols & 7) * (gridDim.x >> 3) + (cols >> 3);
  const int G = a.N / 64, actives = uniform(r.actives);
  const int parts = min(G, (DOWN_WAVES + actives - 1) / actives), units = actives * parts;
  struct Cursor {
    int unit, e, s0, left, c, c1;
  } at, ahead;
  auto open = [&](Cursor& u) __attribute__((always_inline)) {
    if (u.unit >= units) return;
    const int p = u.unit % parts;
    u.e = uniform(r.active[u.unit / parts]);
    u.s0 = uniform(r.first[u.e]);
    u.left = tokens_of(r, u.e);
    u.c = p * G / parts;
    u.c1 = (p + 1) * G / parts;
  };
  auto advance = [&](Cursor& u) __attribute__((always_inline)) {
    if (++u.c < u.c1) return;
    const int p = u.unit % parts;
    u.c = p * G / parts;
    if (u.left > 16 * MT) {
      u.left -= 16 * MT;
      u.s0 += 16 * MT;
      return;
    }
    u.unit += DOWN_WAVES;
    open(u);
  };
  at.unit = wave;
  open(at);
  if (wave < units) {
    ahead = at;
    struct Slot {
      uint2 w;
      uint32_t s, z;
      uint4 x[MT][2];
    } ring[D];
    const uint16_t* hrow[MT];
    auto rows = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        hrow[mt] = a.H + int64_t(ahead.s0 + min(16 * mt + c16, ahead.left - 1)) * a.N + 16 * j;
    };
    rows();
    auto fetch = [&](Slot& sl) __attribute__((always_inline)) {
      const int64_t row = ahead.e * a.down.stride + int64_t(ahead.c) * a.K + 16 * cols;
      sl.w = *reinterpret_cast<const uint2*>(a.down.w.q + row * 32 + uint32_t(32 * c16 + 8 * j));
      sl.s = (a.down.w.s + row)[c16];
      sl.z = (a.down.w.z + row)[c16];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4* const x = reinterpret_cast<const uint4*>(hrow[mt] + 64 * int64_t(ahead.c));
        sl.x[mt][0] = x[0];
        sl.x[mt][1] = x[1];
      }
      const int s0 = ahead.s0, unit = ahead.unit;
      advance(ahead);
      if (ahead.s0 != s0 || ahead.unit != unit) rows();
    };
    v4f acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(ring[d]);
    bool more = true;
    while (more) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (!more) break;
        v8bf b[2];
        operands(ring[d].w, ring[d].s, ring[d].z, true, b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(v8bf, ring[d].x[mt][h]), b[h], acc[mt], 0, 0, 0);
        fetch(ring[d]);
        if (at.c == at.c1 - 1) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int s = 16 * mt + 4 * j + i;
              if (s < at.left) {
                float* const o = out + r.token[at.s0 + s] * 16 + c16;
                *o = fmaf(r.weight[at.s0 + s], acc[mt][i], *o);
              }
            }
            acc[mt] = v4f{0, 0, 0, 0};
          }
        }
        advance(at);
        more = at.unit < units;
      }
    }
  }
  __syncthreads();
  if (tid >= a.T * 16) return;
  float v = 0.f;
  for (int w = 0; w < DOWN_WAVES; ++w) v += sums[w * a.T * 16 + tid];
  a.Y[int64_t(tid >> 4) * a.K + int64_t(cols) * 16 + (tid & 15)] = f32_to_bf16(v);
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
  const int64_t items = std::min(E, T * top) * (N / 32);
  // 32 rows at a time where that many tokens go to an expert
  const bool two = T * top > 16 * E;
  auto up_kernel = act == SVDQ_SILU ? two ? moe_up_kernel<2, SVDQ_SILU> : moe_up_kernel<1, SVDQ_SILU>
                   : two            ? moe_up_kernel<2, SVDQ_GELU>
                                    : moe_up_kernel<1, SVDQ_GELU>;
  hipLaunchKernelGGL(up_kernel, dim3(unsigned(std::min<int64_t>(items, 512))), dim3(64 * UP_WAVES), 0,
                     s, a);
  SVDQ_TRY(check_launch("awq_moe (up)"));
  const size_t lds = size_t(DOWN_WAVES) * size_t(T) * 16 * 4;
  auto down_kernel = two ? moe_down_kernel<2> : moe_down_kernel<1>;
  // (the most that any call asks for: the attribute is the function's, and a host
  // thread with fewer tokens must not lower it between another's two steps)
  SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(down_kernel),
                                     hipFuncAttributeMaxDynamicSharedMemorySize,
                                     DOWN_WAVES * MAX_TOKENS * 16 * 4));
  hipLaunchKernelGGL(down_kernel, dim3(unsigned(K / 16)), dim3(64 * DOWN_WAVES), lds, s, a);
  return check_launch("awq_moe (down)");
}

}  // namespace svdq
