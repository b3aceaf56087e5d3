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
// fp32; the variance is summed from the differences to the mean (a second sum over
// registers, where sum v^2 - mean^2 would lose the digits of a large mean).  x' enters
// the norm as the fp32 sum, before it is rounded to X's type.

#include "block.h"

using namespace svdq_dev;

namespace {

using svdq::Vec;

constexpr int MAX_WAVES = 16;

// V consecutive elements of a row as they lie in memory, fp32 or bf16.  The loads and
// the conversion are apart, so that all loads of a row are in flight together although
// the types are arguments.
template <int V>
struct Raw;
template <>
struct Raw<8> {
  uint4 a, b;
};
template <>
struct Raw<1> {
  uint32_t a;
};

__device__ __forceinline__ void load(Raw<8>& r, const void* p, bool b16, int64_t at) {
  const uint4* const q =
      reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (b16 ? 2 : 4));
  r.a = q[0];
  if (!b16) r.b = q[1];
}
__device__ __forceinline__ void load(Raw<1>& r, const void* p, bool b16, int64_t at) {
  if (b16)
    r.a = static_cast<const uint16_t*>(p)[at];
  else
    r.a = static_cast<const uint32_t*>(p)[at];
}

__device__ __forceinline__ void value(const Raw<8>& r, bool b16, float (&v)[8]) {
  const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
  if (b16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}
__device__ __forceinline__ void value(const Raw<1>& r, bool b16, float (&v)[1]) {
  v[0] = __uint_as_float(b16 ? r.a << 16 : r.a);
}

__device__ __forceinline__ void store(void* p, bool b16, int64_t at, const float (&v)[8]) {
  if (b16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  } else {
    float4* const q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void store(void* p, bool b16, int64_t at, const float (&v)[1]) {
  if (b16)
    static_cast<uint16_t*>(p)[at] = f32_to_bf16(v[0]);
  else
    static_cast<float*>(p)[at] = v[0];
}

// the sum over a wave, in every lane
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value,
                                                    decltype(rows)::value, 0xF, true));
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});   // row_shr 1
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});   // row_shr 2
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});   // row_shr 4
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});   // row_shr 8
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // row_bcast 15
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // row_bcast 31
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums over a workgroup, in every thread.  Each call takes the next of two LDS
// buffers, so that one barrier a call is enough: a wave can write a buffer again only
// past the barrier of the call between, which every wave reaches after its reads.
struct Sums {
  float (*red)[2][MAX_WAVES];
  int waves, wave, turn;

  __device__ __forceinline__ Sums(float (*lds)[2][MAX_WAVES])
      : red(lds), waves(int(blockDim.x) >> 6),
        wave(__builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6)), turn(0) {}

  __device__ __forceinline__ void operator()(float& a, float& b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (waves == 1) return;
    turn ^= 1;
    red[turn][0][wave] = a;
    red[turn][1][wave] = b;
    __syncthreads();
    a = b = 0.f;
    for (int w = 0; w < waves; ++w) {
      a += red[turn][0][w];
      b += red[turn][1][w];
    }
  }
  __device__ __forceinline__ void operator()(float& a) {
    a = wave_sum(a);
    if (waves == 1) return;
    turn ^= 1;
    red[turn][0][wave] = a;
    __syncthreads();
    a = 0.f;
    for (int w = 0; w < waves; ++w) a += red[turn][0][w];
  }
};

// a row's share of a thread: C pieces of V columns, piece c at (c NT + tid) V
template <int V, int C>
struct Row {
  float v[C][V];
};

// v -> n(v); returns 1 / deviation.  Pieces past D hold zeros before and after.
template <int V, int C>
__device__ __forceinline__ float normalize(Row<V, C>& r, const bool (&live)[C], bool layer, int D,
                                           float eps, Sums& sum) {
  const float inv = 1.f / float(D);
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) s += r.v[c][i];
    sum(s);
    const float mean = s * inv;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) r.v[c][i] = live[c] ? r.v[c][i] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(r.v[c][i], r.v[c][i], s);
  sum(s);
  const float rstd = 1.f / sqrtf(fmaf(s, inv, eps));
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[c][i] *= rstd;
  return rstd;
}

template <int V, int C>
__device__ __forceinline__ void norm_row(const svdq::BlockNorm& a, int64_t row, void* X_out,
                                         void* Y, bool y16, Sums& sum) {
  const int64_t image = row / a.rows;
  const int NT = blockDim.x, D = int(a.D);
  bool live[C];
  int col[C];
  Raw<V> x[C], h[C], post[C], gate[C], weight[C], scale[C], shift[C];
  auto vec = [&](Raw<V>& r, const Vec& v, int c) __attribute__((always_inline)) {
    if (v.p && live[c]) load(r, v.p, v.b16, image * v.ld + col[c]);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + int(threadIdx.x)) * V;
    live[c] = col[c] < D;
    if (live[c]) {
      load(x[c], a.X, a.x16, row * D + col[c]);
      if (a.H) load(h[c], a.H, a.h16, row * D + col[c]);
    }
    vec(post[c], a.post, c);
    vec(gate[c], a.gate, c);
    vec(weight[c], a.weight, c);
    vec(scale[c], a.scale, c);
    vec(shift[c], a.shift, c);
  }
  Row<V, C> t, xn;
  if (a.H) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      value(h[c], a.h16, t.v[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) t.v[c][i] = live[c] ? t.v[c][i] : 0.f;
    }
    if (a.post.p) {
      normalize<V, C>(t, live, a.layer, D, a.eps, sum);
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
    value(x[c], a.x16, xn.v[c]);
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
      if (live[c]) store(X_out, a.x16, row * D + col[c], xn.v[c]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) xn.v[c][i] = live[c] ? xn.v[c][i] : 0.f;
  }
  normalize<V, C>(xn, live, a.layer, D, a.eps, sum);
#pragma unroll
  for (int c = 0; c < C; ++c) {
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
    if (live[c]) store(Y, y16, row * D + col[c], xn.v[c]);
  }
}

// a row a workgroup, and the rows past the grid in turn
constexpr int64_t MOST_GROUPS = 1 << 20;

template <int V, int C>
__global__ __launch_bounds__(1024) void block_norm_kernel(svdq::BlockNorm a, int64_t M, void* X_out,
                                                          void* Y, bool y16) {
  __shared__ float lds[2][2][MAX_WAVES];
  Sums sum(lds);
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x)
    norm_row<V, C>(a, row, X_out, Y, y16, sum);
}

// ------------------------------------------------------------- backward
// With dn = dY weight (1 + scale) and n = n(x'), r the reciprocal deviation:
//   g  = dX' + r (dn - [mean dn] - n mean(dn n))       (the mean for layer norm)
//   dX = g,  dt = gate g,  dH = dt or the same form of dt post at n(H)
//   dgate = sum g t,  dpost = sum dt n(H),  dweight = sum dY n (1 + scale),
//   dscale = sum dY n weight,  dshift = sum dY         (sums over the rows)
// The statistics are formed again from X and H, which costs no traffic.  A
// workgroup takes rows of one image one after another and sums the vectors' gradients
// in registers; its sums are joined by a second launch in a fixed order.

enum { POST, GATE, WEIGHT, SCALE, SHIFT, VECTORS };

template <int V, int C>
__global__ __launch_bounds__(1024) void block_norm_grad_kernel(svdq::BlockNorm a,
                                                               svdq::BlockNormGrad g) {
  __shared__ float lds[2][2][MAX_WAVES];
  Sums sum(lds);
  const int NT = blockDim.x, D = int(a.D);
  const int64_t image = blockIdx.x / g.parts, part = blockIdx.x % g.parts;
  const int64_t r0 = image * a.rows + part * a.rows / g.parts;
  const int64_t r1 = image * a.rows + (part + 1) * a.rows / g.parts;
  const float inv = 1.f / float(D);
  bool live[C];
  int col[C];
  float vec[VECTORS][C][V], acc[VECTORS][C][V];
  const Vec* const vs[VECTORS] = {&a.post, &a.gate, &a.weight, &a.scale, &a.shift};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + int(threadIdx.x)) * V;
    live[c] = col[c] < D;
#pragma unroll
    for (int k = 0; k < VECTORS; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        vec[k][c][i] = k == SCALE || k == SHIFT ? 0.f : 1.f;
        acc[k][c][i] = 0.f;
      }
      if (k != SHIFT && vs[k]->p && live[c]) {
        Raw<V> raw;
        load(raw, vs[k]->p, vs[k]->b16, image * vs[k]->ld + col[c]);
        value(raw, vs[k]->b16, vec[k][c]);
      }
    }
  }
  for (int64_t row = r0; row < r1; ++row) {
    Raw<V> xr[C], hr[C], dyr[C], dxr[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live[c]) {
        const int64_t at = row * D + col[c];
        load(xr[c], a.X, a.x16, at);
        if (a.H) load(hr[c], a.H, a.h16, at);
        load(dyr[c], g.dY, g.y16, at);
        if (g.dX_out) load(dxr[c], g.dX_out, a.x16, at);
      }
    Row<V, C> t, n, dy;
    float rh = 1.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      value(xr[c], a.x16, n.v[c]);
      value(dyr[c], g.y16, dy.v[c]);
      if (a.H) value(hr[c], a.h16, t.v[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t.v[c][i] = a.H && live[c] ? t.v[c][i] : 0.f;
        n.v[c][i] = live[c] ? n.v[c][i] : 0.f;
        dy.v[c][i] = live[c] ? dy.v[c][i] : 0.f;
      }
    }
    if (a.H && a.post.p) rh = normalize<V, C>(t, live, a.layer, D, a.eps, sum);
    if (a.H)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i)
          n.v[c][i] = fmaf(vec[GATE][c][i], t.v[c][i] * vec[POST][c][i], n.v[c][i]);
    const float r = normalize<V, C>(n, live, a.layer, D, a.eps, sum);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = dy.v[c][i], dn = d * n.v[c][i];
        const float w = vec[WEIGHT][c][i], m = 1.f + vec[SCALE][c][i];
        acc[SHIFT][c][i] += d;
        acc[WEIGHT][c][i] = fmaf(dn, m, acc[WEIGHT][c][i]);
        acc[SCALE][c][i] = fmaf(dn, w, acc[SCALE][c][i]);
        dy.v[c][i] = d * w * m;
        s1 += dy.v[c][i];
        s2 = fmaf(dy.v[c][i], n.v[c][i], s2);
      }
    sum(s1, s2);
    const float m1 = a.layer ? s1 * inv : 0.f, m2 = s2 * inv;
    s1 = s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[V];
      if (g.dX_out)
        value(dxr[c], a.x16, d);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] = live[c] ? d[i] + r * (dy.v[c][i] - m1 - n.v[c][i] * m2) : 0.f;
        const float tv = t.v[c][i], dt = vec[GATE][c][i] * d[i];
        acc[GATE][c][i] = fmaf(d[i], tv * vec[POST][c][i], acc[GATE][c][i]);
        acc[POST][c][i] = fmaf(dt, tv, acc[POST][c][i]);
        dy.v[c][i] = dt * vec[POST][c][i];
        s1 += dy.v[c][i];
        s2 = fmaf(dy.v[c][i], tv, s2);
      }
      if (live[c]) store(g.dX, a.x16, row * D + col[c], d);
    }
    if (!a.H) continue;
    float k1 = 0.f, k2 = 0.f;
    if (a.post.p) {
      sum(s1, s2);
      k1 = a.layer ? s1 * inv : 0.f;
      k2 = s2 * inv;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = rh * (dy.v[c][i] - k1 - t.v[c][i] * k2);
      if (live[c]) store(g.dH, a.h16, row * D + col[c], d);
    }
  }
#pragma unroll
  for (int k = 0; k < VECTORS; ++k)
    if (g.part[k])
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (live[c]) store(g.part[k], false, int64_t(blockIdx.x) * D + col[c], acc[k][c]);
}

// out[i] = sum over the parts of image i (all of them where a vector is shared)
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part, int D,
                                                              int64_t parts,
                                                              float* __restrict__ out) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks = (D + 63) / 64;
  const int64_t image = blockIdx.x / blocks;
  const int col = int(blockIdx.x % blocks) * 64 + lane;
  const float* const p = part + image * parts * D;
  float s = 0.f;
  if (col < D)
    for (int64_t i = wave; i < parts; i += 4) s += p[i * D + col];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < D)
    out[image * D + col] = red[0][lane] + red[1][lane] + (red[2][lane] + red[3][lane]);
}

// threads and pieces of a row.  V = 8 where D and every address allow 16-byte loads
struct Shape {
  int V, C, NT;
};

Shape shape(int64_t D, bool wide) {
  const int V = wide ? 8 : 1;
  const int64_t n = (D + V - 1) / V;
  int C = 1;
  while (C * int64_t(1024) < n) C *= 2;
  return {V, C, int((n + C * 64 - 1) / (C * 64) * 64)};
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool vec_wide(const Vec& v) { return !v.p || (on16(v.p) && v.ld % (v.b16 ? 8 : 4) == 0); }
bool all_wide(const svdq::BlockNorm& a) {
  return a.D % 8 == 0 && on16(a.X) && on16(a.H) && vec_wide(a.post) && vec_wide(a.gate) &&
         vec_wide(a.weight) && vec_wide(a.scale) && vec_wide(a.shift);
}

int64_t grad_parts(int64_t M, int64_t images) {
  const int64_t rows = M / images;
  return std::max<int64_t>(1, std::min(rows, 512 / images));
}

}  // namespace

namespace svdq {

svdq_status launch_join(const float* part, int64_t D, int64_t parts, int64_t each, float* out,
                        hipStream_t s) {
  hipLaunchKernelGGL(join_kernel, dim3(unsigned((D + 63) / 64 * each)), dim3(256), 0, s, part,
                     int(D), parts, out);
  return check_launch("join");
}

svdq_status launch_block_norm(const BlockNorm& a, int64_t M, void* X_out, void* Y, svdq_dtype y_dt,
                              hipStream_t s) {
  const Shape p = shape(a.D, all_wide(a) && on16(X_out) && on16(Y));
  void (*k)(BlockNorm, int64_t, void*, void*, bool) =
      p.V == 8 ? (p.C == 1 ? block_norm_kernel<8, 1> : block_norm_kernel<8, 2>)
      : p.C == 1 ? block_norm_kernel<1, 1>
      : p.C == 2 ? block_norm_kernel<1, 2>
      : p.C == 4 ? block_norm_kernel<1, 4>
      : p.C == 8 ? block_norm_kernel<1, 8>
                 : block_norm_kernel<1, 16>;
  hipLaunchKernelGGL(k, dim3(unsigned(std::min(M, MOST_GROUPS))), dim3(p.NT), 0, s, a, M, X_out, Y,
                     y_dt == SVDQ_BF16);
  return check_launch("block_norm");
}

size_t block_norm_grad_workspace(int64_t M, int64_t D, int64_t images) {
  if (M == 0) return 0;
  return align256(size_t(VECTORS) * size_t(images * grad_parts(M, images)) * size_t(D) * 4);
}

svdq_status launch_block_norm_grad(const BlockNorm& a, BlockNormGrad g, int64_t M, int64_t images,
                                   float* const (&out)[5], void* ws, hipStream_t s) {
  g.parts = M ? grad_parts(M, images) : 0;
  const Vec* const vs[VECTORS] = {&a.post, &a.gate, &a.weight, &a.scale, &a.shift};
  float* at = static_cast<float*>(ws);
  for (int k = 0; k < VECTORS; ++k) {
    g.part[k] = nullptr;
    if (!out[k]) continue;
    const int64_t each = vs[k]->ld ? images : 1;
    if (images * g.parts == each) {       // one workgroup's sums are the gradient
      g.part[k] = out[k];
      continue;
    }
    g.part[k] = at;
    at += images * g.parts * a.D;
  }
  if (M) {
    const Shape p = shape(a.D, all_wide(a) && on16(g.dY) && on16(g.dX_out) && on16(g.dX) &&
                                   on16(g.dH));
    void (*k)(BlockNorm, BlockNormGrad) =
        p.V == 8 ? (p.C == 1 ? block_norm_grad_kernel<8, 1> : block_norm_grad_kernel<8, 2>)
        : p.C == 1 ? block_norm_grad_kernel<1, 1>
        : p.C == 2 ? block_norm_grad_kernel<1, 2>
        : p.C == 4 ? block_norm_grad_kernel<1, 4>
        : p.C == 8 ? block_norm_grad_kernel<1, 8>
                   : block_norm_grad_kernel<1, 16>;
    hipLaunchKernelGGL(k, dim3(unsigned(images * g.parts)), dim3(p.NT), 0, s, a, g);
    SVDQ_TRY(check_launch("block_norm_grad"));
  }
  for (int k = 0; k < VECTORS; ++k) {
    if (!out[k] || g.part[k] == out[k]) continue;
    const int64_t each = vs[k]->ld ? images : 1, parts = images * g.parts / each;
    SVDQ_TRY(launch_join(g.part[k], a.D, parts, each, out[k], s));
  }
  return SVDQ_OK;
}

}  // namespace svdq
