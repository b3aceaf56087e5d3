// Norms before and after a block, fused with its gate and residual sum (gfx950):
//
//   t  = H, or n(H) * post          (post norm)
//   x' = X + gate * t
//   Y  = n(x') * weight * (1 + scale) + shift
//
// n(v) = (v - mean v) / sqrt(var v + eps) (layer norm) or v / sqrt(mean v^2 + eps)
// (RMS norm) along a row of D.  gate, scale and shift are one vector for all rows or
// one per image (a run of M / images rows); post and weight likewise.
//
// One workgroup takes one row at a time and keeps it in registers between the
// sums, so every matrix is read and written once: the bound is memory.  Sums are
// fp32, but for the mean's, which is 64 bits wide: an error of the mean of a few units of
// its last place is in every n of the row, r times it, and no small one where the mean is
// large against the deviation; and 2^14 equal values sum up exactly, so that their
// differences are zeros.  The variance is summed from the differences to the mean (a
// second sum over registers, where sum v^2 - mean^2 would lose the digits of a large
// mean).  x' enters the norm as the fp32 sum, before it is rounded to X's type.
//
// Measured: 9216 rows of 4096, layer norm, gate, scale and shift, bf16: 302 MB in 56-61 us,
// 5.0-5.4 TB/s (a large copy: 5.3); with a post norm 73: two sums more in a row's chain.
// 333 rows of 5455, an fp32 stream, RMS norms before and after, 9.7-10.4 us, 2.4-2.6 TB/s:
// all rows are resident at once, one or two workgroups of 11 waves to a compute unit, and
// nothing follows that would hide a row's chain of loads, two sums over the workgroup and
// stores (one row takes 4.4, 128 rows 5.6, 256 7.6, 512 11.0).  One row of 4096 2.5-3 us, a
// launch.  Rows of a few hundred values leave most lanes idle: 9216 rows of 64 take 10.5 us
// as 9216 of 512 do.
//
// The 64-bit sum of the mean adds about 0.1 us to each sum of a row's chain: 9216 rows of
// 4096 60.5 -> 61.3 us, with a post norm 68.6 -> 73.2, 4608 rows of 8192 with one 101 ->
// 111, and within 2% in the backward pass from 2048 columns and 9216 rows on.  The adds in
// a thread cost nothing of that (in fp32, or in pairs: the same times); the row operations
// and the turn through LDS do.

#include "block.h"

using namespace svdq_dev;

namespace {

using svdq::Vec;

constexpr int MAX_WAVES = 16;

// How a row is cut into pieces of V elements: all threads have as many; or not, with the
// last piece moved back to end with the row where D is no multiple of V, its first
// elements counting as absent (a branch for a short piece would cost every load: 9216
// rows of 4096 78 us against 60); or D < V, one thread with element-wise accesses.
enum Tail { FULL, MOVED, TINY };

// Types of the matrices: bits X16, H16, Y16 if they are known at compile time (loads
// behind branches on the type wait for one another), ANY if not.
constexpr int ANY = -1;
enum { X16 = 1, H16 = 2, Y16 = 4 };

template <int T>
__device__ __forceinline__ bool type16(int bit, bool b16) {
  return T == ANY ? b16 : (T & bit) != 0;
}

// V consecutive elements of a row as they lie in memory, fp32 or bf16.  The loads and
// the conversion are apart, so that all loads of a row are in flight together.  Addresses
// are multiples of the element only (the target's accesses of 8 and 16 bytes take them).
template <int V>
struct Raw {
  uint32_t w[V];
};

// A thread's share of a row: C pieces of V columns from col[c] on, of which the first
// skip[c] are absent (V: all, nothing is loaded or stored)
template <int V, int C, int TAIL>
struct Cut {
  int col[C], skip[C], D;

  __device__ __forceinline__ explicit Cut(int D) : D(D) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      col[c] = (c * int(blockDim.x) + int(threadIdx.x)) * V;
      const int left = D - col[c];
      skip[c] = left <= 0 ? V : 0;
      if (TAIL == MOVED && left > 0 && left < V) {
        skip[c] = V - left;
        col[c] = D - V;
      }
    }
  }
  __device__ __forceinline__ bool any(int c) const { return TAIL == FULL || skip[c] < V; }
  __device__ __forceinline__ bool in(int c, int i) const {
    return TAIL == FULL ? true : TAIL == MOVED ? i >= skip[c] : col[c] + i < D;
  }
};

template <int V, int C, int TAIL>
__device__ __forceinline__ void load(Raw<V>& r, const Cut<V, C, TAIL>& cut, int c, const void* p,
                                     bool b16, int64_t first) {
  if (!cut.any(c)) return;
  const uint8_t* const q = static_cast<const uint8_t*>(p) + (first + cut.col[c]) * (b16 ? 2 : 4);
  if (TAIL != TINY) {
    // (b16 may be known here; if not, the first half is loaded alike for both types)
    if (__builtin_constant_p(b16) && !b16) {
      __builtin_memcpy(r.w, q, 4 * V);
    } else {
      __builtin_memcpy(r.w, q, 2 * V);
      if (!b16) __builtin_memcpy(r.w + V / 2, q + 2 * V, 2 * V);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t v = 0;
      if (cut.in(c, i)) {
        if (b16)
          v = reinterpret_cast<const uint16_t*>(q)[i];
        else
          v = reinterpret_cast<const uint32_t*>(q)[i];
      }
      if (!b16)
        r.w[i] = v;
      else if (i & 1)
        r.w[i / 2] |= v << 16;
      else
        r.w[i / 2] = v;
    }
  }
}

template <int V>
__device__ __forceinline__ void value(const Raw<V>& r, bool b16, float (&v)[V]) {
  if (b16) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      v[i] = __uint_as_float(r.w[i / 2] << 16);
      v[i + 1] = __uint_as_float(r.w[i / 2] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}

// (Ordinary stores.  Non-temporal ones make the kernel alone up to a fifth faster, 9216 rows of
// 2048 31.0 -> 25.4 us, but the product that reads its output loses more: norm, product and
// product on 4608 rows of 4096 together 335 us and 341 so, on 64 rows 34.8 and 36.3.)
template <int V, int C, int TAIL>
__device__ __forceinline__ void store(const Cut<V, C, TAIL>& cut, int c, void* p, bool b16,
                                      int64_t first, const float (&v)[V]) {
  if (!cut.any(c)) return;
  const int64_t at = first + cut.col[c];
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V; i += 2) w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
  if (TAIL == FULL || (TAIL == MOVED && cut.skip[c] == 0)) {
    if (b16)
      __builtin_memcpy(static_cast<uint16_t*>(p) + at, w, 2 * V);
    else
      __builtin_memcpy(static_cast<float*>(p) + at, v, 4 * V);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!cut.in(c, i)) continue;
      if (b16)
        static_cast<uint16_t*>(p)[at + i] = uint16_t(w[i / 2] >> 16 * (i & 1));
      else
        static_cast<float*>(p)[at + i] = v[i];
    }
  }
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, true));
}

// the sum over each 16 lanes, in their last one (row_shr 1, 2, 4, 8)
__device__ __forceinline__ float row_sum(float v) {
  return add_dpp<0x118>(add_dpp<0x114>(add_dpp<0x112>(add_dpp<0x111>(v))));
}

// the same in 64 bits
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, ROWS, 0xF, true));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b >> 32)), CTRL, ROWS, 0xF, true));
  return v + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double row_sum(double v) {
  return add_dpp<0x118>(add_dpp<0x114>(add_dpp<0x112>(add_dpp<0x111>(v))));
}
__device__ __forceinline__ double lane_of(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b)), l));
  const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b >> 32)), l));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// the sum over a wave, in every lane (row_bcast 15 and 31 join the rows)
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x143, 0xC>(add_dpp<0x142, 0xA>(row_sum(v)));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
  return lane_of(add_dpp<0x143, 0xC>(add_dpp<0x142, 0xA>(row_sum(v))), 63);
}

// Sums over a workgroup, in every thread: of the waves, then of the waves' sums, which 16
// lanes read.  Each call takes the next of two LDS buffers, so that one barrier a call is
// enough: a wave can write a buffer again only past the barrier of the call between,
// which every wave reaches after its reads.
struct Sums {
  float (*red)[2][MAX_WAVES];
  int waves, wave, lane, turn;

  __device__ __forceinline__ explicit Sums(float (*lds)[2][MAX_WAVES])
      : red(lds), waves(int(blockDim.x) >> 6),
        wave(__builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6)), lane(int(threadIdx.x) & 63),
        turn(0) {}

  // lane 15 and lane 31: the sums of the first and the second set
  __device__ __forceinline__ float read() {
    const float v = red[turn][(lane >> 4) & 1][lane & 15];
    return row_sum((lane & 15) < waves ? v : 0.f);
  }
  static __device__ __forceinline__ float from(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
  }
  __device__ __forceinline__ void operator()(float& a, float& b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (waves == 1) return;
    turn ^= 1;
    red[turn][0][wave] = a;
    red[turn][1][wave] = b;
    __syncthreads();
    const float v = read();
    a = from(v, 15);
    b = from(v, 31);
  }
  __device__ __forceinline__ void operator()(float& a) {
    a = wave_sum(a);
    if (waves == 1) return;
    turn ^= 1;
    red[turn][0][wave] = a;
    __syncthreads();
    a = from(read(), 15);
  }
  // (the halves of a wave's sum in the two sets)
  __device__ __forceinline__ void operator()(double& a) {
    a = wave_sum(a);
    if (waves == 1) return;
    turn ^= 1;
    const uint64_t b = __builtin_bit_cast(uint64_t, a);
    uint32_t(*const w)[MAX_WAVES] = reinterpret_cast<uint32_t(*)[MAX_WAVES]>(red[turn]);
    w[0][wave] = uint32_t(b);
    w[1][wave] = uint32_t(b >> 32);
    __syncthreads();
    const int i = lane & 15;
    const uint64_t v = uint64_t(w[1][i]) << 32 | w[0][i];
    a = lane_of(row_sum(i < waves ? __builtin_bit_cast(double, v) : 0.), 15);
  }
};

template <int V, int C>
struct Row {
  float v[C][V];
};

// v -> n(v); returns 1 / deviation.  Elements past D hold zeros before and after.
template <int V, int C, int TAIL>
__device__ __forceinline__ float normalize(Row<V, C>& r, const Cut<V, C, TAIL>& cut, bool layer, int D,
                                           double per, float eps, Sums& sum) {
  const float inv = 1.f / float(D);
  if (layer) {
    double s = 0.;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) s += double(r.v[c][i]);
    sum(s);
    // s / D: the product with the reciprocal, and what it leaves of s (a sum of D equal
    // values gives the value); in two fp32 numbers, of which v - hi takes the first exactly
    // where the mean is large against the differences
    const double q = s * per, mean = fma(fma(-q, double(D), s), per, q);
    const float hi = float(mean), lo = float(mean - double(hi));
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) r.v[c][i] = cut.in(c, i) ? (r.v[c][i] - hi) - lo : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(r.v[c][i], r.v[c][i], s);
  sum(s);
  // (the hardware's reciprocal root, 1 ulp, where it is not subnormal)
  const float var = fmaf(s, inv, eps);
  const float rstd = var < 0x1p-100f ? 1.f / sqrtf(var) : __builtin_amdgcn_rsqf(var);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[c][i] *= rstd;
  return rstd;
}

template <int V, int C, int TAIL, int T>
__device__ __forceinline__ void norm_row(const svdq::BlockNorm& a, int64_t row, void* X_out,
                                         void* Y, bool y16, Sums& sum) {
  const int64_t image = a.images > 1 ? row / a.rows : 0;
  const int D = int(a.D);
  const Cut<V, C, TAIL> cut(D);
  const bool x16 = type16<T>(X16, a.x16), h16 = type16<T>(H16, a.h16);
  Raw<V> x[C], h[C], post[C], gate[C], weight[C], scale[C], shift[C];
  auto vec = [&](Raw<V>& r, const Vec& v, int c) __attribute__((always_inline)) {
    if (v.p) load(r, cut, c, v.p, v.b16, image * v.ld);
  };
  // (all at once while registers last)
  auto behind = [&](int c) __attribute__((always_inline)) {
    vec(weight[c], a.weight, c);
    vec(scale[c], a.scale, c);
    vec(shift[c], a.shift, c);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load(x[c], cut, c, a.X, x16, row * D);
    if (a.H) load(h[c], cut, c, a.H, h16, row * D);
    vec(post[c], a.post, c);
    vec(gate[c], a.gate, c);
    if (C == 1) behind(c);
  }
  Row<V, C> t, xn;
  if (a.H) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      value(h[c], h16, t.v[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) t.v[c][i] = cut.in(c, i) ? t.v[c][i] : 0.f;
    }
    if (a.post.p) {
      normalize(t, cut, a.layer, D, a.per, a.eps, sum);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[V];
        value(post[c], a.post.b16, f);
#pragma unroll
        for (int i = 0; i < V; ++i) t.v[c][i] *= f[i];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    value(x[c], x16, xn.v[c]);
    if (a.H) {
      if (a.gate.p) {
        float f[V];
        value(gate[c], a.gate.b16, f);
#pragma unroll
        for (int i = 0; i < V; ++i) xn.v[c][i] = fmaf(f[i], t.v[c][i], xn.v[c][i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) xn.v[c][i] += t.v[c][i];
      }
      store(cut, c, X_out, x16, row * D, xn.v[c]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) xn.v[c][i] = cut.in(c, i) ? xn.v[c][i] : 0.f;
  }
  normalize(xn, cut, a.layer, D, a.per, a.eps, sum);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (C > 1) behind(c);
    float f[V];
    if (a.weight.p) {
      value(weight[c], a.weight.b16, f);
#pragma unroll
      for (int i = 0; i < V; ++i) xn.v[c][i] *= f[i];
    }
    if (a.scale.p) {
      value(scale[c], a.scale.b16, f);
#pragma unroll
      for (int i = 0; i < V; ++i) xn.v[c][i] *= 1.f + f[i];
    }
    if (a.shift.p) {
      value(shift[c], a.shift.b16, f);
#pragma unroll
      for (int i = 0; i < V; ++i) xn.v[c][i] += f[i];
    }
    store(cut, c, Y, y16, row * D, xn.v[c]);
  }
}

// a row a workgroup, and the rows past the grid in turn
constexpr int64_t MOST_GROUPS = 1 << 20;

template <int V, int C, int TAIL, int T>
__global__ __launch_bounds__(1024) void block_norm_kernel(svdq::BlockNorm a, int64_t M, void* X_out,
                                                          void* Y, bool y16) {
  __shared__ __align__(16) float lds[2][2][MAX_WAVES];
  Sums sum(lds);
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x)
    norm_row<V, C, TAIL, T>(a, row, X_out, Y, y16, sum);
}

// ------------------------------------------------------------- backward
// With dn = dY weight (1 + scale) and n = n(x'), r the reciprocal deviation:
//   g  = dX' + r (dn - [mean dn] - n mean(dn n))       (the mean for layer norm)
//   dX = g,  dt = gate g,  dH = dt or the same form of dt post at n(H)
//   dgate = sum g t,  dpost = sum dt n(H),  dweight = sum dY n (1 + scale),
//   dscale = sum dY n weight,  dshift = sum dY         (sums over the rows)
// The statistics are formed again from X and H, which costs no traffic.
//
// A workgroup takes rows of one image one after another.  Along them the vectors are
// constant, so x' and g need only their products weight (1 + scale) and gate post, and
// three sums a column, A = sum dY n, B = sum g n(H) (or g H) and S = sum dY, hold all
// five gradients: dweight = (1 + scale) A, dscale = weight A, dgate = post B, dpost =
// gate B, dshift = S.  The next row's loads are in flight while one is worked on.  The
// workgroups' sums are joined, and multiplied, by a second launch in a fixed order.
//
// Measured: 9216 rows of 4096, post norm and all five gradients, bf16: 453 MB in 102-104 us,
// 4.4 TB/s, and 8 us for the join.  Between memory and the chain of a row: two or four
// sums over the workgroup follow one another in each row, and the registers of a row,
// the next row and the column sums leave two workgroups a compute unit to hide
// them.  (Five column sums
// spilled: 436 us with them; 175 with three; 111 with the sums over the workgroup in row
// operations of the lanes and the switched-off parts compiled out.)  20 rows of 2048 take
// 4.5 us and the join 3.8.

enum { POST, GATE, WEIGHT, SCALE, SHIFT, VECTORS };

template <int V, int C, int TAIL>
__device__ __forceinline__ void vector(const Vec& v, const Cut<V, C, TAIL>& cut, int64_t image, int c,
                                       float none, float (&out)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = none;
  if (v.p && cut.any(c)) {
    Raw<V> raw;
    load(raw, cut, c, v.p, v.b16, image * v.ld);
    value(raw, v.b16, out);
  }
}

// LONG: rows of more than 8192, in 1024 threads, where 128 registers a thread do not hold
// the two factors too: they lie in LDS (with them in registers 2304 rows of 12288 took 1.8
// times as long, in 512 threads of four pieces 3 times).  The rest does not fit either: of
// x', t, dY, dX' and three sums of 16 columns each the compiler spills 86 to 218 registers,
// 250 to 450 bytes of scratch a lane, fewest for whole rows in bf16.  That traffic is what
// these rows take: everything in use, bf16, 2304 rows of 12288 262-290 us and the join 12 (340
// MB, 64 us at a copy's rate), of 16384 305 and 14, 4096 of 9216 380 and 10; in fp32, or with
// an odd end, 12288 columns 375-390.  The forms for 4097 to 8192 columns with an odd end and
// some one-piece forms of fp32 or unknown types spill up to 9 (fewer than 8 columns: 25).

template <int V, int C, int TAIL, int T, bool LAYER, bool POST_NORM, bool LONG>
__global__ __launch_bounds__(LONG ? 1024 : 512, C == 1 || LONG ? 4 : 2) void block_norm_grad_kernel(
    svdq::BlockNorm a, svdq::BlockNormGrad g) {
  __shared__ __align__(16) float lds[2][2][MAX_WAVES];
  extern __shared__ __align__(16) float factors[];   // LONG: [2][C][threads][V]
  Sums sum(lds);
  const int D = int(a.D);
  const int64_t image = blockIdx.x / g.parts, part = blockIdx.x % g.parts;
  const int64_t r0 = image * a.rows + part * a.rows / g.parts;
  const int64_t r1 = image * a.rows + (part + 1) * a.rows / g.parts;
  const float inv = 1.f / float(D);
  const Cut<V, C, TAIL> cut(D);
  // B's factor and the norm's: gate post, weight (1 + scale)
  constexpr int GP = 0, WM = 1;
  Row<V, C> held[LONG ? 1 : 2], accA, accB, accS;
  auto place = [&](int which, int c) __attribute__((always_inline)) {
    return reinterpret_cast<float4*>(factors + ((which * C + c) * int(blockDim.x) + int(threadIdx.x)) * V);
  };
  auto factor = [&](int which, int c, float (&f)[V]) __attribute__((always_inline)) {
    if constexpr (LONG) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 v = place(which, c)[i / 4];
        f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = held[which].v[c][i];
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float u[V], v[V];
    auto keep = [&](int which) __attribute__((always_inline)) {
      if constexpr (LONG) {
#pragma unroll
        for (int i = 0; i < V; i += 4) place(which, c)[i / 4] = make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) held[which].v[c][i] = u[i];
      }
    };
    vector(a.gate, cut, image, c, 1.f, u);
    vector(a.post, cut, image, c, 1.f, v);
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] *= v[i];
    keep(GP);
    vector(a.weight, cut, image, c, 1.f, u);
    vector(a.scale, cut, image, c, 0.f, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] *= 1.f + v[i];
      accA.v[c][i] = accB.v[c][i] = accS.v[c][i] = 0.f;
    }
    keep(WM);
  }
  const bool x16 = type16<T>(X16, a.x16), h16 = type16<T>(H16, a.h16), y16 = type16<T>(Y16, g.y16);
  Raw<V> xr[C], hr[C], dyr[C], dxr[C];
  // the row's loads, and what they bring: elements past D are zeros
  auto fetch_in = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load(xr[c], cut, c, a.X, x16, row * D);
      if (a.H) load(hr[c], cut, c, a.H, h16, row * D);
    }
  };
  auto fetch_dy = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) load(dyr[c], cut, c, g.dY, y16, row * D);
  };
  auto fetch_dx = [&](int64_t row) __attribute__((always_inline)) {
    if (g.dX_out)
#pragma unroll
      for (int c = 0; c < C; ++c) load(dxr[c], cut, c, g.dX_out, x16, row * D);
  };
  auto take = [&](Row<V, C>& v, const Raw<V> (&raw)[C], bool given, bool b16)
      __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (given)
        value(raw[c], b16, v.v[c]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) v.v[c][i] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) v.v[c][i] = cut.in(c, i) ? v.v[c][i] : 0.f;
    }
  };
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    fetch_in(row);
    fetch_dy(row);
    fetch_dx(row);
  };
  // (a long row's gradients come when they are needed, and nothing of the next one)
  if (!LONG) fetch(r0);
  for (int64_t row = r0; row < r1; ++row) {
    Row<V, C> t, n, dy, d;
    if (LONG) fetch_in(row);
    take(n, xr, true, x16);
    take(t, hr, a.H != nullptr, h16);
    if (!LONG) {
      take(dy, dyr, true, y16);
      take(d, dxr, g.dX_out != nullptr, x16);
      fetch(min(row + 1, r1 - 1));
    }
    float rh = 1.f;
    if (POST_NORM) rh = normalize(t, cut, LAYER, D, a.per, a.eps, sum);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[V];
      factor(GP, c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) n.v[c][i] = fmaf(f[i], t.v[c][i], n.v[c][i]);
    }
    if (LONG) fetch_dy(row);
    const float r = normalize(n, cut, LAYER, D, a.per, a.eps, sum);
    if (LONG) take(dy, dyr, true, y16);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[V];
      factor(WM, c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        accS.v[c][i] += dy.v[c][i];
        accA.v[c][i] = fmaf(dy.v[c][i], n.v[c][i], accA.v[c][i]);
        dy.v[c][i] *= f[i];
        s1 += dy.v[c][i];
        s2 = fmaf(dy.v[c][i], n.v[c][i], s2);
      }
    }
    if (LONG) fetch_dx(row);
    sum(s1, s2);
    if (LONG) take(d, dxr, g.dX_out != nullptr, x16);
    const float m1 = LAYER ? s1 * inv : 0.f, m2 = s2 * inv;
    s1 = s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d.v[c][i] += r * (dy.v[c][i] - m1 - n.v[c][i] * m2);
        d.v[c][i] = cut.in(c, i) ? d.v[c][i] : 0.f;
        accB.v[c][i] = fmaf(d.v[c][i], t.v[c][i], accB.v[c][i]);
      }
      store(cut, c, g.dX, x16, row * D, d.v[c]);
      float f[V];
      factor(GP, c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d.v[c][i] *= f[i];
        s1 += d.v[c][i];
        s2 = fmaf(d.v[c][i], t.v[c][i], s2);
      }
    }
    if (!a.H) continue;
    float k1 = 0.f, k2 = 0.f;
    if (POST_NORM) {
      sum(s1, s2);
      k1 = LAYER ? s1 * inv : 0.f;
      k2 = s2 * inv;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < V; ++i) d.v[c][i] = rh * (d.v[c][i] - k1 - t.v[c][i] * k2);
      store(cut, c, g.dH, h16, row * D, d.v[c]);
    }
  }
  // each gradient is a sum times the vector it shares its product with: here where no
  // other workgroup has part in it, else in the join
  auto put = [&](float* to, const Row<V, C>& acc, const Vec& other, float none, float add)
      __attribute__((always_inline)) {
    if (!to) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[V];
      vector(other, cut, image, c, none, f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = acc.v[c][i] * (f[i] + add);
      store(cut, c, to, false, int64_t(blockIdx.x) * D, f);
    }
  };
  const Vec one{nullptr, 0, false};
  put(g.grad[POST], accB, a.gate, 1.f, 0.f);
  put(g.grad[GATE], accB, a.post, 1.f, 0.f);
  put(g.grad[WEIGHT], accA, a.scale, 0.f, 1.f);
  put(g.grad[SCALE], accA, a.weight, 1.f, 0.f);
  put(g.grad[SHIFT], accS, one, 1.f, 0.f);
  put(g.sums[0], accA, one, 1.f, 0.f);
  put(g.sums[1], accB, one, 1.f, 0.f);
  put(g.sums[2], accS, one, 1.f, 0.f);
}

constexpr int JOIN_WAVES = 8;

// 64 columns and 8 waves a workgroup; every wave adds its share of the parts, one after
// the other, and the waves' sums meet in LDS.  The fixed order is what two calls with the
// same bits need (atomics on the gradients would be one launch).
// 512 parts of 4096 columns in five sums 8.4 us (16 waves 10.2, 4 waves 9.2), 72 parts of
// 12288 5.3 (7.0, 5.3), 20 parts of 2048 3.8 (3.7, 4.4).
__global__ __launch_bounds__(64 * JOIN_WAVES) void join_kernel(svdq::Joins j, int64_t total, int D) {
  __shared__ float red[JOIN_WAVES][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int across = (D + 63) / 64;
  for (int64_t block = blockIdx.x; block < total; block += gridDim.x) {
    int64_t b = block;
    int k = 0;
    while (k + 1 < j.count && b >= j.each[k] * across) b -= j.each[k++] * across;
    const int64_t image = b / across, n = j.each[k] == 1 ? j.images * j.parts : j.parts;
    const int col = int(b % across) * 64 + lane;
    const Vec f = j.factor[k];
    auto factor = [&](int64_t i) __attribute__((always_inline)) {
      if (!f.p) return 1.f;
      const int64_t at = i * f.ld + col;
      return j.plus[k] + (f.b16 ? bf16_to_f32(static_cast<const uint16_t*>(f.p)[at])
                                : static_cast<const float*>(f.p)[at]);
    };
    // where the factor changes along the sum, image by image
    const bool vary = f.p && f.ld && j.each[k] == 1 && j.images > 1;
    // (no parts: no factors either, of which one may be infinite)
    const int64_t each = vary ? j.parts : n, runs = n == 0 ? 0 : vary ? j.images : 1;
    float s = 0.f;
    const float* p = j.from[k] + image * n * D + col;
    if (col < D && vary && j.parts < j.images) {
      // many images: the waves take them in turn, eight at a time.  The steps that follow one
      // another are images / 64 times parts here and images times parts / 64 below.
      // The whole backward pass on 4608 rows of 4096, every gradient, so and in the order
      // below: 4608 images 494 us and 3470, 512 95 and 327, 64 and 128 within 5%.
      for (int64_t r = wave; r < runs; r += 8 * JOIN_WAVES) {
        float t[8], g[8];
        int64_t at[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          at[q] = min(r + JOIN_WAVES * q, runs - 1);
          g[q] = factor(at[q]);
          t[q] = 0.f;
        }
        for (int64_t i = 0; i < each; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q) t[q] += p[(at[q] * each + i) * D];
#pragma unroll
        for (int q = 0; q < 8; ++q) s += r + JOIN_WAVES * q < runs ? t[q] * g[q] : 0.f;
      }
    } else if (col < D) {
      for (int64_t r = 0; r < runs; ++r, p += each * D) {
        float t = 0.f;
        int64_t i = wave;
        for (; i + 7 * JOIN_WAVES < each; i += 8 * JOIN_WAVES) {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = p[(i + JOIN_WAVES * q) * D];
          t += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        for (; i < each; i += JOIN_WAVES) t += p[i * D];
        s += vary ? t * factor(r) : t;
      }
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < D) {
      for (int w = 1; w < JOIN_WAVES; ++w) s += red[w][lane];
      j.to[k][image * D + col] = vary || n == 0 ? s : s * factor(image);
    }
    __syncthreads();
  }
}

// threads and pieces of a row: more pieces than one a thread beyond `most` threads
struct Shape {
  int C, NT;
  Tail tail;
};

constexpr int V = 8;                     // elements of a piece
constexpr int NORM_THREADS = 1024, GRAD_THREADS = 512;

Shape shape(int64_t D, int most) {
  const int64_t n = (D + V - 1) / V;
  int C = 1;
  while (C * int64_t(most) < n) C *= 2;
  const int NT = int((n + C * 64 - 1) / (C * 64) * 64);
  return {C, NT, D < V ? TINY : int64_t(C) * NT * V == D ? FULL : MOVED};
}

// The types that a model's stream meets are known to the kernel: all bf16, an fp32
// stream with bf16 or fp32 blocks.  Others take ANY, and so do rows of two pieces a thread,
// forward from 8193 columns on and backward from 4097, but for whole bf16 rows of more than
// 8192 backward: forms of their own for these are not built, nor measured against ANY.
// With it, everything in use, bf16: backward 7372 rows of 5120 134 us and the join 14, 4608
// of 8192 109 and 12 (86 at a copy's rate); forward 2304 of 12288 76 (43).
template <int TAIL>
auto norm_of(int C, int types) {
  if (C > 1) return block_norm_kernel<V, 2, TAIL, ANY>;
  return types == (X16 | H16) ? block_norm_kernel<V, 1, TAIL, X16 | H16>
         : types == H16       ? block_norm_kernel<V, 1, TAIL, H16>
         : types == 0         ? block_norm_kernel<V, 1, TAIL, 0>
                              : block_norm_kernel<V, 1, TAIL, ANY>;
}

template <int C, int TAIL, int T, bool LONG = false>
auto grad_of(bool layer, bool post) {
  return layer ? post ? block_norm_grad_kernel<V, C, TAIL, T, true, true, LONG>
                      : block_norm_grad_kernel<V, C, TAIL, T, true, false, LONG>
         : post ? block_norm_grad_kernel<V, C, TAIL, T, false, true, LONG>
                : block_norm_grad_kernel<V, C, TAIL, T, false, false, LONG>;
}
auto grad_of(const Shape& p, int types, bool layer, bool post) {
  if (p.NT > GRAD_THREADS)
    return p.tail != FULL                ? grad_of<2, MOVED, ANY, true>(layer, post)
           : types == (X16 | H16 | Y16) ? grad_of<2, FULL, X16 | H16 | Y16, true>(layer, post)
                                         : grad_of<2, FULL, ANY, true>(layer, post);
  if (p.C == 2)
    return p.tail == FULL ? grad_of<2, FULL, ANY>(layer, post) : grad_of<2, MOVED, ANY>(layer, post);
  if (p.tail == TINY) return grad_of<1, TINY, ANY>(layer, post);
  if (p.tail == MOVED)
    return types == (X16 | H16 | Y16) ? grad_of<1, MOVED, X16 | H16 | Y16>(layer, post)
                                      : grad_of<1, MOVED, ANY>(layer, post);
  return types == (X16 | H16 | Y16) ? grad_of<1, FULL, X16 | H16 | Y16>(layer, post)
         : types == (H16 | Y16)     ? grad_of<1, FULL, H16 | Y16>(layer, post)
         : types == Y16             ? grad_of<1, FULL, Y16>(layer, post)
         : types == 0               ? grad_of<1, FULL, 0>(layer, post)
                                    : grad_of<1, FULL, ANY>(layer, post);
}

// (a missing H has X's type: no kernel for it alone)
int types_of(const svdq::BlockNorm& a, bool y16) {
  const bool h16 = a.H ? a.h16 : a.x16;
  return (a.x16 ? X16 : 0) | (h16 ? H16 : 0) | (y16 ? Y16 : 0);
}

// (two pieces a thread of 512 threads, beyond that two of up to 1024)
Shape grad_shape(int64_t D) { return shape(D, D > 2 * GRAD_THREADS * V ? 1024 : GRAD_THREADS); }

// Workgroups an image: 16 waves to a compute unit in all, and at most 1024 workgroups, which
// leaves rows of up to 1024 columns 8 waves and up to 512 columns 4 (9216 rows of 64 take 20
// us and the join 8, of 512 26 in all)
int64_t grad_parts(int64_t M, int64_t D, int64_t images) {
  const int64_t rows = M / images, groups = 256 * (1024 / grad_shape(D).NT);
  return std::max<int64_t>(1, std::min(rows, std::min<int64_t>(groups, 1024) / images));
}

}  // namespace

namespace svdq {

svdq_status launch_joins(const Joins& j, int64_t D, hipStream_t s) {
  int64_t blocks = 0;
  for (int k = 0; k < j.count; ++k) blocks += (D + 63) / 64 * j.each[k];
  if (!blocks) return SVDQ_OK;
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(std::min(blocks, MOST_GROUPS))),
                     dim3(64 * JOIN_WAVES), 0, s, j, blocks, int(D));
  return check_launch("join");
}

svdq_status launch_block_norm(const BlockNorm& a, int64_t M, void* X_out, void* Y, svdq_dtype y_dt,
                              hipStream_t s) {
  const Shape p = shape(a.D, NORM_THREADS);
  const int t = types_of(a, false);
  auto k = p.tail == TINY    ? block_norm_kernel<V, 1, TINY, ANY>
           : p.tail == MOVED ? norm_of<MOVED>(p.C, t)
                             : norm_of<FULL>(p.C, t);
  hipLaunchKernelGGL(k, dim3(unsigned(std::min(M, MOST_GROUPS))), dim3(p.NT), 0, s, a, M, X_out, Y,
                     y_dt == SVDQ_BF16);
  return check_launch("block_norm");
}

size_t block_norm_grad_workspace(int64_t M, int64_t D, int64_t images) {
  if (M == 0) return 0;
  return align256(size_t(3) * size_t(images * grad_parts(M, D, images)) * size_t(D) * 4);
}

svdq_status launch_block_norm_grad(const BlockNorm& a, BlockNormGrad g, int64_t M, int64_t images,
                                   float* const (&out)[5], void* ws, hipStream_t s) {
  g.parts = M ? grad_parts(M, a.D, images) : 0;
  const int64_t groups = images * g.parts;
  const Vec* const vs[VECTORS] = {&a.post, &a.gate, &a.weight, &a.scale, &a.shift};
  // the sum of each gradient, and the vector it is multiplied by
  constexpr int SUM[VECTORS] = {1, 1, 0, 0, 2};
  const Vec factor[VECTORS] = {a.gate, a.post, a.scale, a.weight, {nullptr, 0, false}};
  float* at = static_cast<float*>(ws);
  Joins j{};
  j.parts = g.parts;
  j.images = images;
  for (int k = 0; k < 3; ++k) g.sums[k] = nullptr;
  for (int k = 0; k < VECTORS; ++k) {
    g.grad[k] = nullptr;
    if (!out[k]) continue;
    const int64_t each = vs[k]->ld ? images : 1;
    if (groups == each) {                 // one workgroup's sums are the gradient
      g.grad[k] = out[k];
      continue;
    }
    float*& sum = g.sums[SUM[k]];
    if (!sum) {
      sum = at;
      at += groups * a.D;
    }
    j.add(sum, out[k], each, factor[k], k == WEIGHT ? 1.f : 0.f);
  }
  if (M) {
    const Shape p = grad_shape(a.D);
    auto k = grad_of(p, types_of(a, g.y16), a.layer, a.post.p != nullptr);
    // (the most that any D asks for: the attribute is the function's, and a host thread
    // with a smaller one must not lower it between another's two steps)
    const size_t lds = p.NT > GRAD_THREADS ? size_t(2) * p.C * p.NT * V * 4 : 0;
    if (lds)
      SVDQ_CHECK_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                         hipFuncAttributeMaxDynamicSharedMemorySize,
                                         2 * 2 * 1024 * V * 4));
    hipLaunchKernelGGL(k, dim3(unsigned(images * g.parts)), dim3(p.NT), lds, s, a, g);
    SVDQ_TRY(check_launch("block_norm_grad"));
  }
  return launch_joins(j, a.D, s);
}

}  // namespace svdq
