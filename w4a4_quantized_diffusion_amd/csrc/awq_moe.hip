// A mixture-of-experts layer on AWQ W4A16 experts for few tokens (gfx950):
//
//   e_j, p_j = the top largest of softmax(logits[t]) (ties to the lower expert)
//   Y[t] = sum_j p_j (act(X[t] Wg_e^T) * (X[t] Wu_e^T)) Wd_e^T,   e = e_j
//
// Wg, Wu [E][N, K], Wd [E][K, N] in the AWQ format.  Two launches: the first forms
// H = act(G) * U for every chosen (token, expert) pair, a slot, the second the
// down-projections and their weighted sum; a third adds the sums of slices, where there
// are some.  Every workgroup of the first finds the choices of all tokens in LDS from the
// logits (at most 64 x 256), about a microsecond, where a launch of its own would cost two
// to three, and leaves them to the second.  Slots are sorted by expert, so that each
// expert's weights are read once for all of its tokens.
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

// The routing
struct __attribute__((aligned(16))) Route {
  uint32_t mask[MAX_EXPERTS][2];       // the tokens that chose an expert
  float weight[MAX_SLOTS];             // of a slot
  uint16_t first[MAX_EXPERTS];         // an expert's first slot
  uint8_t active[MAX_EXPERTS];         // experts with tokens, in order
  uint8_t token[MAX_SLOTS];            // of a slot
  int actives;
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
  int S;                  // slices of the down-projections
  float* part;            // their sums [S][T][K], if there are more than one
  Route* route;           // what the first launch found, for the second
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

// from LDS to memory, or back
__device__ __forceinline__ void copy_route(const Route& from, Route& to) {
  static_assert(sizeof(Route) % 16 == 0, "whole pieces");
  for (int i = threadIdx.x; i < int(sizeof(Route) / 16); i += blockDim.x)
    reinterpret_cast<uint4*>(&to)[i] = reinterpret_cast<const uint4*>(&from)[i];
}

// [T][top]
struct Choices {
  uint8_t expert[MAX_SLOTS];
  float p[MAX_SLOTS];
};

// The choices of the tokens, 16 lanes to a token, expert e in lane e % 16; NV values a
// lane (E <= 16 NV).  A lane keeps the token's choice with its number.
template <int NV>
__device__ __forceinline__ void choose(const Moe& a, Route& r, Choices& ch) {
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
    ch.expert[i] = uint8_t(choice);
    ch.p[i] = p;
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
__device__ __forceinline__ void route(const Moe& a, Route& r, Choices& ch) {
  const int tid = threadIdx.x, NT = blockDim.x;
  if (a.T > 1) {
    for (int i = tid; i < 2 * MAX_EXPERTS; i += NT) r.mask[i >> 1][i & 1] = 0;
    __syncthreads();
  } else if (tid == 0) {
    r.actives = a.top;
  }
  if (a.E <= 16)
    choose<1>(a, r, ch);
  else if (a.E <= 32)
    choose<2>(a, r, ch);
  else if (a.E <= 64)
    choose<4>(a, r, ch);
  else if (a.E <= 128)
    choose<8>(a, r, ch);
  else
    choose<16>(a, r, ch);
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
    const int t = i / a.top, e = ch.expert[i];
    // tokens below t in the expert's mask
    const uint32_t lo = t < 32 ? (1u << t) - 1 : 0xFFFFFFFFu, hi = t < 32 ? 0 : (1u << (t - 32)) - 1;
    const int s = r.first[e] + __popc(r.mask[e][0] & lo) + __popc(r.mask[e][1] & hi);
    r.token[s] = uint8_t(t);
    r.weight[s] = ch.p[i];
  }
  __syncthreads();
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Keeps a lane's offset apart from the uniform part of an address, which the compiler
// would fold into a 64-bit sum a lane (no instruction)
__device__ __forceinline__ void opaque(uint32_t& v) { asm volatile("" : "+v"(v)); }

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
// A workgroup's 8 waves take the chunks of K in turn, D of them at a time, and their sums
// meet in LDS.  The workgroups go on from item to item with the next item's loads in
// flight.  (One token runs through the code once: a loop that also unrolled the ends of
// the items took 12 us instead of 9 for it, most of that waiting for instructions.)
//
// One token of 4 experts with N 1024 is 128 items: a workgroup each on half of the compute
// units.
//
// Measured: 61 tokens, 6 of 40 experts, 4096 x 1408: 260 MB of codes and scales in 67-72
// us, 3.6-3.9 TB/s.  The vector units are busy 57% of the cycles, with 2.4-3 instructions
// a code for the dequantization and the routing of operands; a copy of the kernel that only
// loads takes 55 us, and what is left between is the two not overlapping fully.  Three and four
// chunks ahead, 4 or 16 waves a workgroup and 6 waves a SIMD gain nothing; a workgroup per
// item instead of 512 that go on takes 97 us.

constexpr int UP_WAVES = 8;

template <int MT, int ACT>
__global__ __launch_bounds__(64 * UP_WAVES, 4) void moe_up_kernel(Moe a) {
  constexpr int D = 2;
  __shared__ Route r;
  __shared__ Choices ch;
  __shared__ float red[UP_WAVES][MT][2][2][4][64];   // [wave][rows][column parity][G, U][e][lane]
  route(a, r, ch);
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
  if (blockIdx.x == 0)
    copy_route(r, *a.route);
  if (start >= end) return;
  // D steps of an item's slots s0 .. s0 + left - 1
  struct Turn {
    int item, e, block, s0, left, step;
  };
  auto open = [&](Turn& t) __attribute__((always_inline)) {
    t.e = uniform(r.active[t.item / blocks]);
    t.block = t.item % blocks;
    t.s0 = uniform(r.first[t.e]);
    t.left = tokens_of(r, t.e);
  };
  // addresses are a uniform base and a lane's 32-bit offset in bytes (X is at most 64 x
  // 2^22 elements)
  uint32_t xoff[MT];
  auto rows = [&](const Turn& t) __attribute__((always_inline)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      xoff[mt] = 2 * uint32_t(r.token[t.s0 + min(16 * mt + c16, t.left - 1)]) * uint32_t(a.K) + 32 * j;
  };
  uint32_t woff = 64 * c16 + 8 * j, soff = 4 * c16;
  struct Slot {
    uint2 w[2][2];                       // gate, up; column parity
    uint32_t s[2], z[2];                 // of both columns
    uint4 x[MT][2];
  } ring[D];
  // every slot is always loaded (past the last chunk with the last one's data), so that
  // the number of loads in flight is fixed
  auto fetch = [&](const Turn& t, int d, Slot& sl) __attribute__((always_inline)) {
    const int c = min(wave + UP_WAVES * (t.step + d), G - 1);
    const int64_t row = t.e * a.gate.stride + int64_t(c) * a.N + 32 * t.block;
    opaque(woff);
    opaque(soff);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const svdq::AwqWeight& w = i ? a.up.w : a.gate.w;
      const uint8_t* const q = w.q + row * 32;
#pragma unroll
      for (int p = 0; p < 2; ++p)
        sl.w[i][p] = *reinterpret_cast<const uint2*>(q + 32 * p + woff);
      sl.s[i] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(w.s + row) + soff);
      sl.z[i] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(w.z + row) + soff);
    }
    const uint8_t* const x = reinterpret_cast<const uint8_t*>(a.X + 64 * int64_t(c));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      sl.x[mt][0] = *reinterpret_cast<const uint4*>(x + xoff[mt]);
      sl.x[mt][1] = *reinterpret_cast<const uint4*>(x + 16 + xoff[mt]);
    }
  };
  v4f acc[MT][2][2];
  Turn at;
  at.item = start;
  at.step = 0;
  open(at);
  rows(at);
#pragma unroll
  for (int d = 0; d < D; ++d) {
    fetch(at, d, ring[d]);
    // (slot by slot, here and below: the waits count the loads behind a slot's)
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[mt][p][t] = v4f{0, 0, 0, 0};
  while (true) {
    // the turn behind this one: the same slots, the item's next, or the next item's
    // (none: this one again, whose loads are not used)
    Turn next = at;
    const bool last = at.step + D >= steps;
    next.step = last ? 0 : at.step + D;
    if (last) {
      if (at.left > 16 * MT) {
        next.left -= 16 * MT;
        next.s0 += 16 * MT;
      } else {
        next.item += stride;
        if (next.item < end) open(next);
      }
      rows(next);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Slot& sl = ring[d];
      const bool live = wave + UP_WAVES * (at.step + d) < G;
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
      fetch(next, d, sl);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (last) {
      // the waves' sums in order
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) red[wave][mt][p][t][e][lane] = acc[mt][p][t][e];
            acc[mt][p][t] = v4f{0, 0, 0, 0};
          }
      lds_barrier();
      // wave e of four (of each tile of rows): rows 4 j + e, both columns
      const int mt = MT == 1 ? 0 : wave >> 2, e = wave & 3, row = 16 * mt + 4 * j + e;
      if (wave < 4 * MT && row < at.left) {
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
      if (next.item >= end) return;
      lds_barrier();
    }
    at = next;
  }
}

// ---------------------------------------------------- the down-projections
// A workgroup owns 16 CT columns of Y and one of S slices of the active experts' chunks.
// Its 16 waves share them evenly: a wave takes a run of them, D at a time, adds each
// expert's part to the tokens' sums, a set of them per wave in LDS, and the sets are
// joined in order.  A wave goes on from expert to expert with the next one's loads in
// flight.  With S > 1 a third launch adds the slices' sums (the workgroup of a column
// block that ends last could, but its fences write the L2 back and took 9 us).
//
// Measured: 61 tokens as above 130 MB in 42-45 us, 3.0 TB/s, and 4-5 for the sums; one token
// 5.7-6.8 us, in 128 workgroups for K 2048.  A copy that only loads takes 30 us for the 61;
// the rest is the dequantization, an expert's sums in LDS and the fewer bytes in flight at
// their turn.

constexpr int DOWN_WAVES = 16;
constexpr int MAX_SLICES = 8;

template <int MT, int CT>
__global__ __launch_bounds__(64 * DOWN_WAVES) void moe_down_kernel(Moe a) {
  // (with 32 columns 3, 4 and 6 take up to 4 us more for the 61 tokens)
  constexpr int D = MT * CT == 1 ? 4 : 2;
  constexpr int W = 16 * CT;
  __shared__ Route r;
  extern __shared__ __align__(16) float sums[];     // [wave][T][W]
  copy_route(*a.route, r);
  const int tid = threadIdx.x, lane = tid & 63, j = lane >> 4, c16 = lane & 15;
  const int wave = uniform(tid >> 6);
  float* const out = sums + wave * a.T * W;
  for (int i = lane; i < a.T * W; i += 64) out[i] = 0.f;
  __syncthreads();
  // the slices of a column block one behind the other, the blocks of an XCD in a run
  int group = blockIdx.x;
  if ((gridDim.x & 7) == 0) group = (group & 7) * (gridDim.x >> 3) + (group >> 3);
  const int slice = group % a.S, cols = group / a.S;
  const int G = a.N / 64, total = uniform(r.actives) * G, shares = DOWN_WAVES * a.S;
  const int share = slice * DOWN_WAVES + wave;
  const int p0 = int(int64_t(share) * total / shares), p1 = int(int64_t(share + 1) * total / shares);
  // D chunks from c on of a piece c0 .. c1 - 1 of expert number i, slots s0 .. s0 + left -
  // 1; `rest` chunks lie behind the piece
  struct Turn {
    int i, e, s0, left, c0, c, c1, rest;
  };
  auto open = [&](Turn& t) __attribute__((always_inline)) {
    t.e = uniform(r.active[t.i]);
    t.s0 = uniform(r.first[t.e]);
    t.left = tokens_of(r, t.e);
    t.c = t.c0;
    t.c1 = min(G, t.c0 + t.rest);
    t.rest -= t.c1 - t.c0;
  };
  if (p0 < p1) {
    Turn at;
    at.i = p0 / G;
    at.c0 = p0 - at.i * G;
    at.rest = p1 - p0;
    open(at);
    struct Slot {
      uint2 w[CT];
      uint32_t s, z;
      uint4 x[MT][2];
    } ring[D];
    // (a piece's rows of H: at most 64 x 2^22 elements)
    uint32_t hoff[MT];
    auto rows = [&](const Turn& t) __attribute__((always_inline)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        hoff[mt] = 2 * uint32_t(min(16 * mt + c16, t.left - 1)) * uint32_t(a.N) + 32 * j;
    };
    uint32_t woff = 32 * CT * c16 + 8 * j, soff = 2 * CT * c16;
    auto fetch = [&](const Turn& t, int d, Slot& sl) __attribute__((always_inline)) {
      const int c = min(t.c + d, t.c1 - 1);
      const int64_t row = t.e * a.down.stride + int64_t(c) * a.K + W * cols;
      opaque(woff);
      opaque(soff);
      const uint8_t* const s8 = reinterpret_cast<const uint8_t*>(a.down.w.s + row);
      const uint8_t* const z8 = reinterpret_cast<const uint8_t*>(a.down.w.z + row);
#pragma unroll
      for (int p = 0; p < CT; ++p)
        sl.w[p] = *reinterpret_cast<const uint2*>(a.down.w.q + row * 32 + 32 * p + woff);
      if constexpr (CT == 1) {
        sl.s = *reinterpret_cast<const uint16_t*>(s8 + soff);
        sl.z = *reinterpret_cast<const uint16_t*>(z8 + soff);
      } else {
        sl.s = *reinterpret_cast<const uint32_t*>(s8 + soff);
        sl.z = *reinterpret_cast<const uint32_t*>(z8 + soff);
      }
      const uint8_t* const h = reinterpret_cast<const uint8_t*>(a.H + int64_t(t.s0) * a.N + 64 * int64_t(c));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        sl.x[mt][0] = *reinterpret_cast<const uint4*>(h + hoff[mt]);
        sl.x[mt][1] = *reinterpret_cast<const uint4*>(h + 16 + hoff[mt]);
      }
    };
    v4f acc[MT][CT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int p = 0; p < CT; ++p) acc[mt][p] = v4f{0, 0, 0, 0};
    rows(at);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      fetch(at, d, ring[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
    while (true) {
      // the turn behind this one: the same piece, the expert's next slots, or the next
      // expert (none: this one again, whose loads are not used)
      Turn next = at;
      const bool last = at.c + D >= at.c1;
      bool more = true;
      next.c += D;
      if (last) {
        next.c = at.c0;
        if (at.left > 16 * MT) {
          next.left -= 16 * MT;
          next.s0 += 16 * MT;
        } else if (at.rest) {
          ++next.i;
          next.c0 = 0;
          open(next);
        } else {
          more = false;
        }
        rows(next);
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        Slot& sl = ring[d];
#pragma unroll
        for (int p = 0; p < CT; ++p) {
          v8bf b[2];
          operands(sl.w[p], p ? sl.s >> 16 : sl.s & 0xFFFF, p ? sl.z >> 16 : sl.z & 0xFFFF,
                   at.c + d < at.c1, b);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[mt][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(v8bf, sl.x[mt][h]), b[h], acc[mt][p], 0, 0, 0);
        }
        fetch(next, d, sl);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (last) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // (all reads first)
          int to[4];
          float w[4], o[4][CT];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int s = at.s0 + min(16 * mt + 4 * j + i, at.left - 1);
            to[i] = r.token[s] * W + CT * c16;
            w[i] = r.weight[s];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < CT; ++p) o[i][p] = out[to[i] + p];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * mt + 4 * j + i < at.left)
#pragma unroll
              for (int p = 0; p < CT; ++p) out[to[i] + p] = fmaf(w[i], acc[mt][p][i], o[i][p]);
#pragma unroll
          for (int p = 0; p < CT; ++p) acc[mt][p] = v4f{0, 0, 0, 0};
        }
        if (!more) break;
      }
      at = next;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * W; i += 64 * DOWN_WAVES) {
    float v = 0.f;
    for (int w = 0; w < DOWN_WAVES; ++w) v += sums[w * a.T * W + i];
    const int64_t at = int64_t(i / W) * a.K + int64_t(cols) * W + i % W;
    if (a.S == 1)
      a.Y[at] = f32_to_bf16(v);
    else
      a.part[int64_t(slice) * a.T * a.K + at] = v;
  }
}

// Y from the slices' sums, in order; 4 columns per thread
__global__ __launch_bounds__(64) void moe_sum_kernel(const float* __restrict__ part, int S,
                                                     int64_t total, uint16_t* __restrict__ Y) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= total) return;
  v4f v[MAX_SLICES], p = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < MAX_SLICES; ++q)
    v[q] = reinterpret_cast<const v4f*>(part)[int64_t(min(q, S - 1)) * total + i];
#pragma unroll
  for (int q = 0; q < MAX_SLICES; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] += q < S ? v[q][e] : 0.f;
  reinterpret_cast<uint2*>(Y)[i] = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
}

struct Plan {
  bool two_rows, two_columns;
  int S;
};

// Measured, us.  16 rows at a time against 32 (tokens an expert): 64 tokens, 64 experts, 8
// each, 2048 x 768 (8) 61 / 67; 61 tokens, 40, 6, 4096 x 1408 (9) 116 / 125; 64 tokens, 16,
// 4, 4096 x 1024 (16) 64 / 53; 64 tokens, 8, 2, 4096 x 2048 (16) 65 / 53.
// 16 columns of the down-projection a workgroup against 32 with slices: one token, 4 of 32
// experts, 2048 x 1024 15.1 / 18.0 (the third launch), 2 of 8, 8192 x 2048 29.6 / 28.4 (K
// of 8192 needs no slices); 8 tokens, 2 of 8, 1024 x 512 14.4 / 13.5; 16 tokens, 8 of 64,
// 2048 x 768 64 / 51; 64 tokens, 8 of 256, 2048 x 256 89 / 76.
Plan plan(int64_t T, int64_t E, int64_t top, int64_t K) {
  Plan p{};
  p.two_rows = T * top > 12 * E;
  p.two_columns = T > 1 || K >= 8192;
  p.S = 1;
  if (p.two_columns)
    while (p.S < MAX_SLICES && p.S * (K / 32) < 256) p.S *= 2;
  return p;
}

size_t h_bytes(int64_t T, int64_t top, int64_t N) {
  return svdq::align256(size_t(T) * size_t(top) * size_t(N) * 2);
}
}  // namespace

namespace svdq {

size_t awq_moe_workspace(int64_t T, int64_t E, int64_t top, int64_t K, int64_t N) {
  const Plan p = plan(T, E, top, K);
  return align256(sizeof(Route)) + h_bytes(T, top, N) +
         (p.S == 1 ? 0 : align256(size_t(p.S) * size_t(T) * size_t(K) * 4));
}

svdq_status launch_awq_moe(const uint16_t* X, const void* logits, bool l16, int64_t T, int64_t E,
                           int64_t top, int64_t K, int64_t N, AwqWeight gate, AwqWeight up,
                           AwqWeight down, svdq_act act, bool renorm, uint16_t* Y, int32_t* ids,
                           float* weights, void* ws, hipStream_t s) {
  const int64_t rows = K * N / 64;
  const Plan p = plan(T, E, top, K);
  uint8_t* const h = static_cast<uint8_t*>(ws) + align256(sizeof(Route));
  float* const part = reinterpret_cast<float*>(h + h_bytes(T, top, N));
  const Moe a{X, logits, l16, renorm, int(T), int(E), int(top), int(K), int(N),
              {gate, rows}, {up, rows}, {down, rows}, reinterpret_cast<uint16_t*>(h), Y, ids,
              weights, p.S, part, static_cast<Route*>(ws)};
  const int64_t items = std::min(E, T * top) * (N / 32);
  auto up_kernel = act == SVDQ_SILU
                       ? p.two_rows ? moe_up_kernel<2, SVDQ_SILU> : moe_up_kernel<1, SVDQ_SILU>
                   : p.two_rows ? moe_up_kernel<2, SVDQ_GELU>
                                : moe_up_kernel<1, SVDQ_GELU>;
  hipLaunchKernelGGL(up_kernel, dim3(unsigned(std::min<int64_t>(items, 512))), dim3(64 * UP_WAVES), 0,
                     s, a);
  SVDQ_TRY(check_launch("awq_moe (up)"));
  const int W = p.two_columns ? 32 : 16;
  const size_t lds = size_t(DOWN_WAVES) * size_t(T) * size_t(W) * 4;
  // (one token has no two rows of an expert)
  auto down_kernel = !p.two_columns ? moe_down_kernel<1, 1>
                     : p.two_rows   ? moe_down_kernel<2, 2>
                                    : moe_down_kernel<1, 2>;
  // (the most that any call asks for: the attribute is the function's, and a host
  // thread with fewer tokens must not lower it between another's two steps)
  if (lds + sizeof(Route) > (64 << 10))
    SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(down_kernel),
                                       hipFuncAttributeMaxDynamicSharedMemorySize,
                                       DOWN_WAVES * MAX_TOKENS * 4 * W));
  hipLaunchKernelGGL(down_kernel, dim3(unsigned(K / W * p.S)), dim3(64 * DOWN_WAVES), lds, s, a);
  SVDQ_TRY(check_launch("awq_moe (down)"));
  if (p.S == 1) return SVDQ_OK;
  const int64_t quads = T * K / 4;
  hipLaunchKernelGGL(moe_sum_kernel, dim3(unsigned((quads + 63) / 64)), dim3(64), 0, s, part, p.S,
                     quads, Y);
  return check_launch("awq_moe (sum)");
}

}  // namespace svdq
