// C ABI front end: argument validation, workspace layout, dispatch, and the
// per-thread error message.  Every check runs before any HIP call.

#include "block.h"

#include <cstdio>
#include <mutex>
#include <string>

namespace svdq {

namespace {
thread_local std::string g_err;
}

void set_error(const std::string& m) { g_err = m; }
void clear_error() { g_err.clear(); }
svdq_status fail(svdq_status st, const std::string& m) {
  g_err = m;
  return st;
}
svdq_status check_launch(const char* what) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SVDQ_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return SVDQ_OK;
}

int cu_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace svdq

using svdq::fail;

namespace {

// every kernel forms row offsets within one K-group as 32-bit integers
constexpr int64_t MAX_DIM = (int64_t(1) << 27) - 1;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

svdq_status check_ptr(const void* p, const char* name, size_t align = 16) {
  if (!p) return fail(SVDQ_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned(p, align))
    return fail(SVDQ_ERR_INVALID_ARG, std::string(name) + " is not " + std::to_string(align) +
                                          "-byte aligned");
  return SVDQ_OK;
}

svdq_status check_dtype(svdq_dtype d, const char* name) {
  if (d != SVDQ_F32 && d != SVDQ_BF16)
    return fail(SVDQ_ERR_INVALID_ARG, std::string(name) + ": unknown dtype");
  return SVDQ_OK;
}

svdq_status check_prec(svdq_precision p) {
  if (p != SVDQ_INT4 && p != SVDQ_NVFP4) return fail(SVDQ_ERR_INVALID_ARG, "unknown precision");
  return SVDQ_OK;
}

svdq_status check_mkr(int64_t M, int64_t K, int32_t rank) {
  if (M < 0 || M > MAX_DIM) return fail(SVDQ_ERR_INVALID_ARG, "M out of range");
  if (K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 64");
  if (rank < 0 || rank > 256 || rank % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "rank must be a multiple of 16 in [0, 256]");
  if (M * K > (int64_t(1) << 40)) return fail(SVDQ_ERR_INVALID_ARG, "M*K too large");
  return SVDQ_OK;
}

// The GEMM kernels cover Y with 256 x 256 tiles, one workgroup each, and
// index tiles with 32-bit integers.
svdq_status check_tiles(int64_t M, int64_t N) {
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (tiles > int64_t(INT32_MAX))
    return fail(SVDQ_ERR_INVALID_ARG, "M x N too large: more than 2^31 - 1 output tiles of 256 x 256");
  return SVDQ_OK;
}

#define TRY(x)                            \
  do {                                    \
    svdq_status st_ = (x);                \
    if (st_ != SVDQ_OK) return st_;       \
  } while (0)

struct Layout {
  size_t codes, scales, lr, total;
};

Layout layout(int64_t M, int64_t K, int32_t rank, svdq_precision prec) {
  Layout l;
  l.codes = 0;
  const size_t codes_b = size_t(M) * size_t(K / 2);
  l.scales = svdq::align256(codes_b);
  const size_t scales_b = prec == SVDQ_INT4 ? size_t(M) * size_t(K / 64) * 4 : size_t(M) * size_t(K / 16);
  l.lr = l.scales + svdq::align256(scales_b);
  l.total = l.lr + svdq::align256(size_t(M) * size_t(rank) * 2);
  return l;
}

}  // namespace

extern "C" {

const char* svdq_last_error(void) { return svdq::g_err.c_str(); }

size_t svdq_workspace_bytes(int64_t M, int64_t K, int32_t rank, svdq_precision prec) {
  if (check_mkr(M, K, rank) != SVDQ_OK || check_prec(prec) != SVDQ_OK) return 0;
  return layout(M, K, rank, prec).total;
}

void svdq_workspace_layout(int64_t M, int64_t K, int32_t rank, svdq_precision prec,
                           size_t* codes_off, size_t* scales_off, size_t* lr_off) {
  Layout l = layout(M, K, rank, prec);
  if (codes_off) *codes_off = l.codes;
  if (scales_off) *scales_off = l.scales;
  if (lr_off) *lr_off = l.lr;
}

svdq_status svdq_act_absmax(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K,
                            float* amax, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_dtype(x_dtype, "x_dtype"));
  if (M < 0 || M > MAX_DIM || K <= 0 || K > MAX_DIM)
    return fail(SVDQ_ERR_INVALID_ARG, "M or K out of range");
  TRY(check_ptr(amax, "amax", 4));
  if (M == 0) return SVDQ_OK;
  TRY(check_ptr(X, "X", x_dtype == SVDQ_F32 ? 4 : 2));
  return svdq::launch_act_absmax(X, x_dtype, M, K, amax, stream);
}

svdq_status svdq_quantize_weights(const float* W, int64_t N, int64_t K, const float* act_amax,
                                  int32_t rank, svdq_precision prec, uint32_t flags,
                                  float* smooth, uint16_t* lora_down, uint16_t* lora_up,
                                  uint8_t* wcodes, void* wscales, float* w_tensor_scale,
                                  float* x_tensor_scale, float* residual, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_prec(prec));
  if (N <= 0 || N > MAX_DIM) return fail(SVDQ_ERR_INVALID_ARG, "N must be positive");
  if (K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 64");
  if (N * K > (int64_t(1) << 33)) return fail(SVDQ_ERR_INVALID_ARG, "N*K too large");
  if (rank < 0 || rank > N || rank > K) return fail(SVDQ_ERR_INVALID_ARG, "rank must be in [0, min(N, K)]");
  if (flags & ~SVDQ_LOWRANK_GIVEN) return fail(SVDQ_ERR_INVALID_ARG, "unknown flags");
  TRY(check_ptr(W, "W", 4));
  if (act_amax) TRY(check_ptr(act_amax, "act_amax", 4));
  TRY(check_ptr(smooth, "smooth", 4));
  if (rank > 0) {
    TRY(check_ptr(lora_down, "lora_down", 2));
    TRY(check_ptr(lora_up, "lora_up", 2));
  }
  TRY(check_ptr(wcodes, "wcodes", 1));
  TRY(check_ptr(wscales, "wscales", prec == SVDQ_INT4 ? 4 : 1));
  if (prec == SVDQ_NVFP4) {
    TRY(check_ptr(w_tensor_scale, "w_tensor_scale", 4));
    TRY(check_ptr(x_tensor_scale, "x_tensor_scale", 4));
  }
  if (residual) TRY(check_ptr(residual, "residual", 4));
  return svdq::quantize_weights_impl(W, N, K, act_amax, rank, prec, flags, smooth, lora_down,
                                     lora_up, wcodes, wscales, w_tensor_scale, x_tensor_scale,
                                     residual, stream);
}

}  // extern "C"

namespace {

// the activation step, with or without GELU applied to X first
svdq_status act_quantize(const void* X, svdq_dtype x_dtype, bool gelu, int64_t M, int64_t K,
                         int32_t rank, svdq_precision prec, const float* smooth,
                         const uint16_t* lora_down, const float* x_tensor_scale,
                         uint8_t* codes, void* scales, uint16_t* LR, hipStream_t stream) {
  TRY(check_dtype(x_dtype, "x_dtype"));
  if (gelu && x_dtype != SVDQ_BF16)
    return fail(SVDQ_ERR_UNSUPPORTED, "the GELU input form takes bf16 activations");
  TRY(check_prec(prec));
  TRY(check_mkr(M, K, rank));
  if (M == 0) return SVDQ_OK;
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(smooth, "smooth"));
  TRY(check_ptr(codes, "codes", 4));
  TRY(check_ptr(scales, "scales", 4));
  if (rank > 0) {
    TRY(check_ptr(lora_down, "lora_down"));
    TRY(check_ptr(LR, "LR"));
  }
  if (prec == SVDQ_NVFP4) {
    TRY(check_ptr(x_tensor_scale, "x_tensor_scale", 4));
    return svdq::launch_act_quant_nvfp4(X, x_dtype, gelu, M, K, rank, smooth, lora_down,
                                        x_tensor_scale, codes, static_cast<uint8_t*>(scales),
                                        LR, stream);
  }
  return svdq::launch_act_quant_int4(X, x_dtype, gelu, M, K, rank, smooth, lora_down, codes,
                                     static_cast<float*>(scales), LR, stream);
}

}  // namespace

extern "C" {

svdq_status svdq_act_quantize(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K,
                              int32_t rank, svdq_precision prec, const float* smooth,
                              const uint16_t* lora_down, const float* x_tensor_scale,
                              uint8_t* codes, void* scales, uint16_t* LR, hipStream_t stream) {
  svdq::clear_error();
  return act_quantize(X, x_dtype, false, M, K, rank, prec, smooth, lora_down, x_tensor_scale,
                      codes, scales, LR, stream);
}

svdq_status svdq_act_quantize_gelu(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K,
                                   int32_t rank, svdq_precision prec, const float* smooth,
                                   const uint16_t* lora_down, const float* x_tensor_scale,
                                   uint8_t* codes, void* scales, uint16_t* LR,
                                   hipStream_t stream) {
  svdq::clear_error();
  return act_quantize(X, x_dtype, true, M, K, rank, prec, smooth, lora_down, x_tensor_scale,
                      codes, scales, LR, stream);
}

svdq_status svdq_gemm_w4a4(const uint8_t* codes, const void* scales, const uint16_t* LR,
                           int64_t M, int64_t K, int64_t N, int32_t rank,
                           svdq_precision prec, const uint8_t* wcodes, const void* wscales,
                           const uint16_t* lora_up, const float* w_tensor_scale,
                           const float* x_tensor_scale, const void* bias,
                           svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype,
                           hipStream_t stream) {
  svdq::clear_error();
  TRY(check_prec(prec));
  TRY(check_mkr(M, K, rank));
  TRY(check_dtype(y_dtype, "y_dtype"));
  if (bias) TRY(check_dtype(bias_dtype, "bias_dtype"));
  if (N <= 0 || N > MAX_DIM || N % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16");
  TRY(check_tiles(M, N));
  if (M == 0) return SVDQ_OK;
  TRY(check_ptr(codes, "codes"));
  TRY(check_ptr(scales, "scales", 4));
  TRY(check_ptr(wcodes, "wcodes"));
  TRY(check_ptr(wscales, "wscales", 4));
  TRY(check_ptr(Y, "Y"));
  if (bias) TRY(check_ptr(bias, "bias", 4));
  if (rank > 0) {
    TRY(check_ptr(LR, "LR"));
    TRY(check_ptr(lora_up, "lora_up"));
  }
  if (prec == SVDQ_NVFP4) {
    TRY(check_ptr(w_tensor_scale, "w_tensor_scale", 4));
    TRY(check_ptr(x_tensor_scale, "x_tensor_scale", 4));
    return svdq::launch_gemm_nvfp4(codes, static_cast<const uint8_t*>(scales), LR, M, K, N,
                                   rank, wcodes, static_cast<const uint8_t*>(wscales), lora_up,
                                   w_tensor_scale, x_tensor_scale, bias, bias_dtype, Y,
                                   y_dtype, stream);
  }
  return svdq::launch_gemm_int4(codes, static_cast<const float*>(scales), LR, M, K, N, rank,
                                wcodes, static_cast<const float*>(wscales), lora_up, bias,
                                bias_dtype, Y, y_dtype, stream);
}

}  // extern "C"

namespace {

svdq_status linear_w4a4(const void* X, svdq_dtype x_dtype, bool gelu, int64_t M, int64_t K,
                        int64_t N, int32_t rank, svdq_precision prec, const float* smooth,
                        const uint16_t* lora_down, const uint16_t* lora_up,
                        const uint8_t* wcodes, const void* wscales,
                        const float* w_tensor_scale, const float* x_tensor_scale,
                        const void* bias, svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  TRY(check_dtype(x_dtype, "x_dtype"));
  if (bias) TRY(check_dtype(bias_dtype, "bias_dtype"));
  if (gelu && x_dtype != SVDQ_BF16)
    return fail(SVDQ_ERR_UNSUPPORTED, "the GELU input form takes bf16 activations");
  TRY(check_prec(prec));
  TRY(check_mkr(M, K, rank));
  if (N <= 0 || N > MAX_DIM || N % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16");
  TRY(check_tiles(M, N));
  if (M == 0) return SVDQ_OK;
  const Layout l = layout(M, K, rank, prec);
  TRY(check_ptr(workspace, "workspace", 256));
  if (workspace_bytes < l.total)
    return fail(SVDQ_ERR_INVALID_ARG, "workspace too small: need " + std::to_string(l.total) +
                                          " bytes");
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(Y, "Y"));
  {
    const uintptr_t w0 = reinterpret_cast<uintptr_t>(workspace), w1 = w0 + l.total;
    const size_t xb = size_t(M) * size_t(K) * (x_dtype == SVDQ_F32 ? 4 : 2);
    const size_t yb = size_t(M) * size_t(N) * (y_dtype == SVDQ_F32 ? 4 : 2);
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(X), y0 = reinterpret_cast<uintptr_t>(Y);
    if ((x0 < w1 && w0 < x0 + xb) || (y0 < w1 && w0 < y0 + yb) || (x0 < y0 + yb && y0 < x0 + xb))
      return fail(SVDQ_ERR_INVALID_ARG, "X, Y and workspace must not overlap");
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TRY(act_quantize(X, x_dtype, gelu, M, K, rank, prec, smooth, lora_down, x_tensor_scale,
                   ws + l.codes, ws + l.scales,
                   rank > 0 ? reinterpret_cast<uint16_t*>(ws + l.lr) : nullptr, stream));
  return svdq_gemm_w4a4(ws + l.codes, ws + l.scales,
                        rank > 0 ? reinterpret_cast<const uint16_t*>(ws + l.lr) : nullptr, M, K,
                        N, rank, prec, wcodes, wscales, lora_up, w_tensor_scale,
                        x_tensor_scale, bias, bias_dtype, Y, y_dtype, stream);
}

}  // namespace

extern "C" {

svdq_status svdq_linear_w4a4(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K, int64_t N,
                             int32_t rank, svdq_precision prec, const float* smooth,
                             const uint16_t* lora_down, const uint16_t* lora_up,
                             const uint8_t* wcodes, const void* wscales,
                             const float* w_tensor_scale, const float* x_tensor_scale,
                             const void* bias, svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  return linear_w4a4(X, x_dtype, false, M, K, N, rank, prec, smooth, lora_down, lora_up, wcodes,
                     wscales, w_tensor_scale, x_tensor_scale, bias, bias_dtype, Y, y_dtype,
                     workspace, workspace_bytes, stream);
}

svdq_status svdq_linear_w4a4_gelu(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K,
                                  int64_t N, int32_t rank, svdq_precision prec,
                                  const float* smooth, const uint16_t* lora_down,
                                  const uint16_t* lora_up, const uint8_t* wcodes,
                                  const void* wscales, const float* w_tensor_scale,
                                  const float* x_tensor_scale, const void* bias,
                                  svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  return linear_w4a4(X, x_dtype, true, M, K, N, rank, prec, smooth, lora_down, lora_up, wcodes,
                     wscales, w_tensor_scale, x_tensor_scale, bias, bias_dtype, Y, y_dtype,
                     workspace, workspace_bytes, stream);
}

}  // extern "C"

// ----------------------------------------------------------- no allocation
// The workspace of svdq_linear_w4a4_noalloc: a fixed device array (each GPU
// the library runs on holds its own copy until the process ends).  Its name
// is only a host-side stand-in; host code uses the device address that
// hipGetSymbolAddress returns for the current device.
namespace {

constexpr size_t SCRATCH_BYTES = size_t(32) << 20;
static __device__ __align__(256) uint8_t scratch[SCRATCH_BYTES];

constexpr int MAX_DEVICES = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[MAX_DEVICES] = {};

// the scratch array's address on the current device, looked up once per device
svdq_status scratch_on_current_device(void** out) {
  int dev = -1;
  SVDQ_CHECK_HIP(hipGetDevice(&dev));
  if (dev < 0 || dev >= MAX_DEVICES) return fail(SVDQ_ERR_UNSUPPORTED, "device index out of range");
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    SVDQ_CHECK_HIP(hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)));
    if (!ptr) return fail(SVDQ_ERR_HIP, "hipGetSymbolAddress returned no address");
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t svdq_noalloc_max_workspace_bytes(void) { return SCRATCH_BYTES; }

svdq_status svdq_linear_w4a4_noalloc(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K,
                                     int64_t N, int32_t rank, svdq_precision prec,
                                     const float* smooth, const uint16_t* lora_down,
                                     const uint16_t* lora_up, const uint8_t* wcodes,
                                     const void* wscales, const float* w_tensor_scale,
                                     const float* x_tensor_scale, const void* bias,
                                     svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype,
                                     hipStream_t stream) {
  svdq::clear_error();
  TRY(check_prec(prec));
  TRY(check_mkr(M, K, rank));
  if (M == 0) return SVDQ_OK;
  const size_t need = layout(M, K, rank, prec).total;
  if (need > SCRATCH_BYTES)
    return fail(SVDQ_ERR_INVALID_ARG, "the workspace of M=" + std::to_string(M) + ", K=" +
                                          std::to_string(K) + ", rank=" + std::to_string(rank) +
                                          " needs " + std::to_string(need) +
                                          " bytes, above the fixed scratch of " +
                                          std::to_string(SCRATCH_BYTES) + " bytes");
  // the usual argument checks of the layer before the first HIP call
  TRY(check_dtype(x_dtype, "x_dtype"));
  TRY(check_dtype(y_dtype, "y_dtype"));
  if (bias) TRY(check_dtype(bias_dtype, "bias_dtype"));
  if (N <= 0 || N > MAX_DIM || N % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16");
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(Y, "Y"));
  void* ws = nullptr;
  TRY(scratch_on_current_device(&ws));
  return linear_w4a4(X, x_dtype, false, M, K, N, rank, prec, smooth, lora_down, lora_up, wcodes,
                     wscales, w_tensor_scale, x_tensor_scale, bias, bias_dtype, Y, y_dtype, ws,
                     SCRATCH_BYTES, stream);
}

svdq_status svdq_fold_lora(const uint16_t* lora_down, const uint16_t* lora_up, int64_t N,
                           int64_t K, int32_t rank, const uint16_t* A, const uint16_t* B,
                           int32_t r_lora, float scale, uint16_t* lora_down_out,
                           uint16_t* lora_up_out, int32_t* rank_out, hipStream_t stream) {
  svdq::clear_error();
  if (N <= 0 || N > MAX_DIM || K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N > 0 and K a positive multiple of 64 required");
  if (rank < 0 || rank % 16 != 0 || rank > 256)
    return fail(SVDQ_ERR_INVALID_ARG, "rank must be a multiple of 16 in [0, 256]");
  if (r_lora <= 0 || r_lora > 256) return fail(SVDQ_ERR_INVALID_ARG, "r_lora must be in [1, 256]");
  const int32_t r_new = (rank + r_lora + 15) / 16 * 16;
  if (r_new > 256) return fail(SVDQ_ERR_INVALID_ARG, "rank + r_lora must stay at most 256");
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f)
    return fail(SVDQ_ERR_INVALID_ARG, "scale must be finite");
  if (!rank_out) return fail(SVDQ_ERR_INVALID_ARG, "rank_out is NULL");
  if (rank > 0) {
    TRY(check_ptr(lora_down, "lora_down", 2));
    TRY(check_ptr(lora_up, "lora_up", 2));
  }
  TRY(check_ptr(A, "A", 2));
  TRY(check_ptr(B, "B", 2));
  TRY(check_ptr(lora_down_out, "lora_down_out", 2));
  TRY(check_ptr(lora_up_out, "lora_up_out", 2));
  {
    // the outputs may not overlap any input or each other
    const size_t e = sizeof(uint16_t);
    const uintptr_t d0 = reinterpret_cast<uintptr_t>(lora_down_out), d1 = d0 + size_t(r_new) * K * e;
    const uintptr_t u0 = reinterpret_cast<uintptr_t>(lora_up_out), u1 = u0 + size_t(N) * r_new * e;
    const struct { const void* p; size_t b; } in[4] = {
        {lora_down, size_t(rank) * K * e}, {lora_up, size_t(N) * rank * e},
        {A, size_t(r_lora) * K * e}, {B, size_t(N) * r_lora * e}};
    bool bad = d0 < u1 && u0 < d1;
    for (const auto& r : in) {
      if (!r.p || r.b == 0) continue;
      const uintptr_t p0 = reinterpret_cast<uintptr_t>(r.p), p1 = p0 + r.b;
      bad = bad || (p0 < d1 && d0 < p1) || (p0 < u1 && u0 < p1);
    }
    if (bad) return fail(SVDQ_ERR_INVALID_ARG, "the outputs must not overlap the inputs or each other");
  }
  TRY(svdq::launch_fold_lora(lora_down, lora_up, N, K, rank, A, B, r_lora, scale, r_new,
                             lora_down_out, lora_up_out, stream));
  *rank_out = r_new;
  return SVDQ_OK;
}

svdq_status awq_quantize_weights(const float* W, int64_t N, int64_t K, int32_t group, uint8_t* q,
                                 uint16_t* scales, uint16_t* zeros, hipStream_t stream) {
  svdq::clear_error();
  if (group != 64) return fail(SVDQ_ERR_UNSUPPORTED, "group must be 64");
  if (N <= 0 || N > MAX_DIM || K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N > 0 and K a positive multiple of 64 required");
  TRY(check_ptr(W, "W", 4));
  TRY(check_ptr(q, "q", 1));
  TRY(check_ptr(scales, "scales", 2));
  TRY(check_ptr(zeros, "zeros", 2));
  return svdq::launch_awq_quant(W, N, K, q, scales, zeros, stream);
}

svdq_status awq_linear_w4a16(const uint16_t* X, int64_t M, int64_t K, int64_t N, int32_t group,
                             const uint8_t* q, const uint16_t* scales, const uint16_t* zeros,
                             const uint16_t* bias, void* Y, svdq_dtype y_dtype,
                             hipStream_t stream) {
  svdq::clear_error();
  if (group != 64) return fail(SVDQ_ERR_UNSUPPORTED, "group must be 64");
  TRY(check_dtype(y_dtype, "y_dtype"));
  if (M < 0 || M > MAX_DIM) return fail(SVDQ_ERR_INVALID_ARG, "M out of range");
  if (K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 64");
  if (N <= 0 || N > MAX_DIM || N % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16");
  TRY(check_tiles(M, N));
  if (M == 0) return SVDQ_OK;
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(q, "q"));
  TRY(check_ptr(scales, "scales", 2));
  TRY(check_ptr(zeros, "zeros", 2));
  TRY(check_ptr(Y, "Y"));
  if (bias) TRY(check_ptr(bias, "bias", 2));
  return svdq::launch_awq_linear(X, M, K, N, q, scales, zeros, bias, Y, y_dtype, stream);
}

}  // extern "C"

// ------------------------------------------------- weight-only operators
namespace {

// a DEVICE operand's extent, for the overlap checks
struct Span {
  const void* p;
  size_t bytes;
  bool out;
};

// no output overlaps an operand or another output
svdq_status check_spans(const Span* v, int n) {
  for (int i = 0; i < n; ++i) {
    if (!v[i].out || !v[i].p || !v[i].bytes) continue;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(v[i].p), a1 = a0 + v[i].bytes;
    for (int j = 0; j < n; ++j) {
      if (j == i || !v[j].p || !v[j].bytes) continue;
      const uintptr_t b0 = reinterpret_cast<uintptr_t>(v[j].p), b1 = b0 + v[j].bytes;
      if (a0 < b1 && b0 < a1)
        return fail(SVDQ_ERR_INVALID_ARG,
                    "outputs and workspace must not overlap the inputs or each other");
    }
  }
  return SVDQ_OK;
}

svdq_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return SVDQ_OK;
  if (have < need)
    return fail(SVDQ_ERR_INVALID_ARG, "workspace too small: need " + std::to_string(need) + " bytes");
  return check_ptr(ws, "workspace", 256);
}

// the tiled kernels form offsets inside a tile of 256 rows as 32-bit byte counts
constexpr int64_t MAX_WIDTH = int64_t(1) << 22;

svdq_status check_mkn(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || M > MAX_DIM) return fail(SVDQ_ERR_INVALID_ARG, "M out of range");
  if (K <= 0 || K > MAX_DIM || K % 64 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "K must be a positive multiple of 64");
  if (N <= 0 || N > MAX_DIM || N % 16 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 16");
  if (K > MAX_WIDTH || N > MAX_WIDTH)
    return fail(SVDQ_ERR_INVALID_ARG, "K and N must be at most 2^22");
  const int64_t most = int64_t(1) << 40;
  if (M * K > most || M * N > most || N * K > most)
    return fail(SVDQ_ERR_INVALID_ARG, "M*K, M*N and N*K must be at most 2^40");
  return SVDQ_OK;
}

svdq_status check_act(svdq_act a) {
  if (a != SVDQ_SILU && a != SVDQ_GELU) return fail(SVDQ_ERR_INVALID_ARG, "unknown activation");
  return SVDQ_OK;
}

svdq_status check_group(int32_t group) {
  if (group != 64) return fail(SVDQ_ERR_UNSUPPORTED, "group must be 64");
  return SVDQ_OK;
}

svdq_status check_awq(const svdq::AwqWeight& w, const char* which) {
  TRY(check_ptr(w.q, (std::string("q") + which).c_str()));
  TRY(check_ptr(w.s, (std::string("scales") + which).c_str()));
  return check_ptr(w.z, (std::string("zeros") + which).c_str());
}

size_t elem(svdq_dtype d) { return d == SVDQ_F32 ? 4 : 2; }

constexpr int64_t A16_ROWS = 64;

}  // namespace

extern "C" {

size_t svdq_linear_w4a16_workspace_bytes(int64_t M, int64_t K, int64_t N, int32_t rank) {
  if (check_mkr(M, K, rank) != SVDQ_OK || check_mkn(M, K, N) != SVDQ_OK || M > A16_ROWS) return 0;
  return svdq::linear_a16_workspace(M, K, N, rank);
}

svdq_status svdq_linear_w4a16(const void* X, svdq_dtype x_dtype, int64_t M, int64_t K, int64_t N,
                              int32_t rank, svdq_precision prec, const float* smooth,
                              const uint16_t* lora_down, const uint16_t* lora_up,
                              const uint8_t* wcodes, const void* wscales,
                              const float* w_tensor_scale, const void* bias,
                              svdq_dtype bias_dtype, void* Y, svdq_dtype y_dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_dtype(x_dtype, "x_dtype"));
  TRY(check_dtype(y_dtype, "y_dtype"));
  if (bias) TRY(check_dtype(bias_dtype, "bias_dtype"));
  TRY(check_prec(prec));
  TRY(check_mkr(M, K, rank));
  TRY(check_mkn(M, K, N));
  if (M > A16_ROWS)
    return fail(SVDQ_ERR_UNSUPPORTED, "svdq_linear_w4a16 takes at most 64 rows");
  if (M == 0) return SVDQ_OK;
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(smooth, "smooth"));
  if (rank > 0) {
    TRY(check_ptr(lora_down, "lora_down"));
    TRY(check_ptr(lora_up, "lora_up"));
  }
  TRY(check_ptr(wcodes, "wcodes"));
  TRY(check_ptr(wscales, "wscales"));
  if (prec == SVDQ_NVFP4) TRY(check_ptr(w_tensor_scale, "w_tensor_scale", 4));
  if (bias) TRY(check_ptr(bias, "bias", elem(bias_dtype)));
  TRY(check_ptr(Y, "Y"));
  const size_t need = svdq::linear_a16_workspace(M, K, N, rank);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t m = M, k = K, n = N, r = rank;
  const Span spans[] = {{X, m * k * elem(x_dtype), false}, {smooth, k * 4, false},
                        {rank ? lora_down : nullptr, r * k * 2, false},
                        {rank ? lora_up : nullptr, r * n * 2, false}, {wcodes, n * k / 2, false},
                        {wscales, n * k / 16, false}, {bias, n * elem(bias_dtype), false},
                        {prec == SVDQ_NVFP4 ? w_tensor_scale : nullptr, 4, false},
                        {Y, m * n * elem(y_dtype), true}, {workspace, need, true}};
  TRY(check_spans(spans, 10));
  return svdq::launch_linear_a16(X, x_dtype, M, K, N, rank, prec, smooth, lora_down, lora_up,
                                 wcodes, wscales, w_tensor_scale, bias, bias_dtype, Y, y_dtype,
                                 workspace, stream);
}

size_t awq_gated_w4a16_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_mkn(M, K, N) != SVDQ_OK) return 0;
  return svdq::awq_gated_workspace(M, K, N);
}

svdq_status awq_gated_w4a16(const uint16_t* X, int64_t M, int64_t K, int64_t N, int32_t group,
                            const uint8_t* q_gate, const uint16_t* scales_gate,
                            const uint16_t* zeros_gate, const uint16_t* bias_gate,
                            const uint8_t* q_up, const uint16_t* scales_up,
                            const uint16_t* zeros_up, const uint16_t* bias_up, svdq_act act,
                            void* H, svdq_dtype h_dtype, uint16_t* G_out, uint16_t* U_out,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_dtype(h_dtype, "h_dtype"));
  TRY(check_act(act));
  TRY(check_mkn(M, K, N));
  TRY(check_tiles(M, 2 * N));
  if (M == 0) return SVDQ_OK;
  const svdq::AwqWeight wg{q_gate, scales_gate, zeros_gate}, wu{q_up, scales_up, zeros_up};
  TRY(check_ptr(X, "X"));
  TRY(check_awq(wg, "_gate"));
  TRY(check_awq(wu, "_up"));
  if (bias_gate) TRY(check_ptr(bias_gate, "bias_gate", 2));
  if (bias_up) TRY(check_ptr(bias_up, "bias_up", 2));
  TRY(check_ptr(H, "H"));
  if (!G_out != !U_out)
    return fail(SVDQ_ERR_INVALID_ARG, "G_out and U_out are given together or not at all");
  if (G_out) {
    TRY(check_ptr(G_out, "G_out"));
    TRY(check_ptr(U_out, "U_out"));
  }
  const size_t need = svdq::awq_gated_workspace(M, K, N);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t m = M, k = K, n = N;
  const Span spans[] = {{X, m * k * 2, false}, {q_gate, n * k / 2, false},
                        {scales_gate, n * k / 32, false}, {zeros_gate, n * k / 32, false},
                        {bias_gate, n * 2, false}, {q_up, n * k / 2, false},
                        {scales_up, n * k / 32, false}, {zeros_up, n * k / 32, false},
                        {bias_up, n * 2, false}, {H, m * n * elem(h_dtype), true},
                        {G_out, m * n * 2, true}, {U_out, m * n * 2, true},
                        {workspace, need, true}};
  TRY(check_spans(spans, 13));
  return svdq::launch_awq_gated(X, M, K, N, wg, wu, bias_gate, bias_up, act, H, h_dtype, G_out,
                                U_out, workspace, stream);
}

size_t awq_gated_w4a16_grad_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_mkn(M, K, N) != SVDQ_OK) return 0;
  return svdq::awq_gated_grad_workspace(M, K, N);
}

svdq_status awq_gated_w4a16_grad(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                 int64_t M, int64_t K, int64_t N, int32_t group,
                                 const uint8_t* q_gate, const uint16_t* scales_gate,
                                 const uint16_t* zeros_gate, const uint8_t* q_up,
                                 const uint16_t* scales_up, const uint16_t* zeros_up,
                                 svdq_act act, uint16_t* dX, uint16_t* dG, uint16_t* dU,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_act(act));
  TRY(check_mkn(M, K, N));
  TRY(check_tiles(M, K));
  if (M == 0) return SVDQ_OK;
  const svdq::AwqWeight wg{q_gate, scales_gate, zeros_gate}, wu{q_up, scales_up, zeros_up};
  TRY(check_ptr(dH, "dH"));
  TRY(check_ptr(G, "G"));
  TRY(check_ptr(U, "U"));
  TRY(check_awq(wg, "_gate"));
  TRY(check_awq(wu, "_up"));
  TRY(check_ptr(dX, "dX"));
  TRY(check_ptr(dG, "dG"));
  TRY(check_ptr(dU, "dU"));
  const size_t need = svdq::awq_gated_grad_workspace(M, K, N);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t m = M, k = K, n = N;
  const Span spans[] = {{dH, m * n * 2, false}, {G, m * n * 2, false}, {U, m * n * 2, false},
                        {q_gate, n * k / 2, false}, {scales_gate, n * k / 32, false},
                        {zeros_gate, n * k / 32, false}, {q_up, n * k / 2, false},
                        {scales_up, n * k / 32, false}, {zeros_up, n * k / 32, false},
                        {dX, m * k * 2, true}, {dG, m * n * 2, true}, {dU, m * n * 2, true},
                        {workspace, need, true}};
  TRY(check_spans(spans, 13));
  return svdq::launch_awq_gated_grad(dH, G, U, M, K, N, wg, wu, act, dX, dG, dU, workspace, stream);
}

size_t awq_linear_w4a16_grad_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_mkn(M, K, N) != SVDQ_OK) return 0;
  return svdq::awq_linear_grad_workspace(M, K, N);
}

svdq_status awq_linear_w4a16_grad(const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                                  int32_t group, const uint8_t* q, const uint16_t* scales,
                                  const uint16_t* zeros, void* dX, svdq_dtype dx_dtype,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_dtype(dx_dtype, "dx_dtype"));
  TRY(check_mkn(M, K, N));
  TRY(check_tiles(M, K));
  if (M == 0) return SVDQ_OK;
  const svdq::AwqWeight w{q, scales, zeros};
  TRY(check_ptr(dY, "dY"));
  TRY(check_awq(w, ""));
  TRY(check_ptr(dX, "dX"));
  const size_t need = svdq::awq_linear_grad_workspace(M, K, N);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t m = M, k = K, n = N;
  const Span spans[] = {{dY, m * n * 2, false}, {q, n * k / 2, false}, {scales, n * k / 32, false},
                        {zeros, n * k / 32, false}, {dX, m * k * elem(dx_dtype), true},
                        {workspace, need, true}};
  TRY(check_spans(spans, 6));
  return svdq::launch_awq_linear_grad(dY, M, K, N, w, dX, dx_dtype, workspace, stream);
}

}  // extern "C"

// ------------------------------------------------- norms around a block
namespace {

// a workgroup holds a row in registers
constexpr int64_t MAX_NORM = 16384;
constexpr int64_t MAX_IMAGES = int64_t(1) << 20;

svdq_status check_norm(int64_t M, int64_t D, int64_t images, svdq_norm kind, float eps) {
  if (M < 0 || M > MAX_DIM) return fail(SVDQ_ERR_INVALID_ARG, "M out of range");
  if (D <= 0) return fail(SVDQ_ERR_INVALID_ARG, "D must be positive");
  if (D > MAX_NORM) return fail(SVDQ_ERR_UNSUPPORTED, "D must be at most 16384");
  if (images <= 0 || images > MAX_IMAGES || M % images != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "images must be in [1, 2^20] and divide M");
  if (kind != SVDQ_LAYER_NORM && kind != SVDQ_RMS_NORM)
    return fail(SVDQ_ERR_INVALID_ARG, "unknown norm");
  if (!(eps >= 0.f && eps <= 3.4e38f))
    return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and not negative");
  return SVDQ_OK;
}

// the vector as the kernels take it, and its extent
svdq_status take_vec(const svdq_vec* v, const char* name, int64_t D, int64_t images, svdq::Vec& out,
                     Span& span) {
  out = {nullptr, 0, false};
  span = {nullptr, 0, false};
  if (!v) return SVDQ_OK;
  const std::string n = name;
  TRY(check_dtype(v->dtype, (n + ".dtype").c_str()));
  TRY(check_ptr(v->data, (n + ".data").c_str(), elem(v->dtype)));
  if (v->ld != 0 && (v->ld < D || v->ld > (int64_t(1) << 40) / images))
    return fail(SVDQ_ERR_INVALID_ARG, n + ".ld must be 0 or at least D");
  out = {v->data, v->ld, v->dtype == SVDQ_BF16};
  const int64_t last = v->ld * (images - 1) + D;
  span = {v->data, size_t(last) * elem(v->dtype), false};
  return SVDQ_OK;
}

const char* const VEC_NAMES[] = {"post", "gate", "weight", "scale", "shift"};

svdq_status take_vecs(const svdq_vec* const (&v)[5], bool block, int64_t D, int64_t images,
                      svdq::BlockNorm& a, Span* spans) {
  svdq::Vec* const to[] = {&a.post, &a.gate, &a.weight, &a.scale, &a.shift};
  for (int i = 0; i < 5; ++i) TRY(take_vec(v[i], VEC_NAMES[i], D, images, *to[i], spans[i]));
  if (!block && (a.post.p || a.gate.p))
    return fail(SVDQ_ERR_INVALID_ARG, "post and gate go with H");
  return SVDQ_OK;
}

}  // namespace

extern "C" {

svdq_status svdq_block_norm(const void* X, svdq_dtype x_dtype, const void* H, svdq_dtype h_dtype,
                            int64_t M, int64_t D, int64_t images, svdq_norm kind, float eps,
                            const svdq_vec* post, const svdq_vec* gate, const svdq_vec* weight,
                            const svdq_vec* scale, const svdq_vec* shift, void* X_out, void* Y,
                            svdq_dtype y_dtype, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_dtype(x_dtype, "x_dtype"));
  if (H) TRY(check_dtype(h_dtype, "h_dtype"));
  TRY(check_dtype(y_dtype, "y_dtype"));
  TRY(check_norm(M, D, images, kind, eps));
  if (M == 0) return SVDQ_OK;
  svdq::BlockNorm a{X, H, x_dtype == SVDQ_BF16, h_dtype == SVDQ_BF16, kind == SVDQ_LAYER_NORM, D,
                    images, M / images, eps, 1. / double(D)};
  Span spans[9];
  TRY(check_ptr(X, "X", elem(x_dtype)));
  TRY(take_vecs({post, gate, weight, scale, shift}, H != nullptr, D, images, a, spans));
  if (!H != !X_out)
    return fail(SVDQ_ERR_INVALID_ARG, "H and X_out are given together or not at all");
  if (H) {
    TRY(check_ptr(H, "H", elem(h_dtype)));
    TRY(check_ptr(X_out, "X_out", elem(x_dtype)));
  }
  TRY(check_ptr(Y, "Y", elem(y_dtype)));
  const size_t n = size_t(M) * size_t(D);
  spans[5] = {X, n * elem(x_dtype), false};
  spans[6] = {H, n * elem(h_dtype), false};
  spans[7] = {X_out, n * elem(x_dtype), true};
  spans[8] = {Y, n * elem(y_dtype), true};
  TRY(check_spans(spans, 9));
  return svdq::launch_block_norm(a, M, X_out, Y, y_dtype, stream);
}

size_t svdq_block_norm_grad_workspace_bytes(int64_t M, int64_t D, int64_t images) {
  if (check_norm(M, D, images, SVDQ_RMS_NORM, 0.f) != SVDQ_OK) return 0;
  return svdq::block_norm_grad_workspace(M, D, images);
}

svdq_status svdq_block_norm_grad(const void* dY, svdq_dtype y_dtype, const void* dX_out,
                                 const void* X, svdq_dtype x_dtype, const void* H,
                                 svdq_dtype h_dtype, int64_t M, int64_t D, int64_t images,
                                 svdq_norm kind, float eps, const svdq_vec* post,
                                 const svdq_vec* gate, const svdq_vec* weight,
                                 const svdq_vec* scale, const svdq_vec* shift, void* dX, void* dH,
                                 float* dpost, float* dgate, float* dweight, float* dscale,
                                 float* dshift, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  svdq::clear_error();
  TRY(check_dtype(y_dtype, "y_dtype"));
  TRY(check_dtype(x_dtype, "x_dtype"));
  if (H || dH) TRY(check_dtype(h_dtype, "h_dtype"));
  TRY(check_norm(M, D, images, kind, eps));
  svdq::BlockNorm a{X, H, x_dtype == SVDQ_BF16, h_dtype == SVDQ_BF16, kind == SVDQ_LAYER_NORM, D,
                    images, M / images, eps, 1. / double(D)};
  const svdq::BlockNormGrad g{dY, dX_out, dX, dH, y_dtype == SVDQ_BF16};
  Span spans[17];
  // (without rows there is no H to go by)
  TRY(take_vecs({post, gate, weight, scale, shift}, H != nullptr || M == 0, D, images, a, spans));
  float* const out[5] = {dpost, dgate, dweight, dscale, dshift};
  const svdq::Vec* const vs[] = {&a.post, &a.gate, &a.weight, &a.scale, &a.shift};
  for (int i = 0; i < 5; ++i) {
    spans[5 + i] = {nullptr, 0, true};
    if (!out[i]) continue;
    const std::string n = std::string("d") + VEC_NAMES[i];
    if (!vs[i]->p)
      return fail(SVDQ_ERR_INVALID_ARG, n + " is asked for without " + VEC_NAMES[i]);
    TRY(check_ptr(out[i], n.c_str()));
    spans[5 + i].p = out[i];
    spans[5 + i].bytes = size_t(vs[i]->ld ? images : 1) * size_t(D) * 4;
  }
  const size_t n = size_t(M) * size_t(D), need = svdq::block_norm_grad_workspace(M, D, images);
  if (M) {
    TRY(check_ptr(dY, "dY", elem(y_dtype)));
    TRY(check_ptr(X, "X", elem(x_dtype)));
    TRY(check_ptr(dX, "dX", elem(x_dtype)));
    if (!H != !dH) return fail(SVDQ_ERR_INVALID_ARG, "H and dH are given together or not at all");
    if (H) {
      TRY(check_ptr(H, "H", elem(h_dtype)));
      TRY(check_ptr(dH, "dH", elem(h_dtype)));
    }
    if (dX_out) TRY(check_ptr(dX_out, "dX_out", elem(x_dtype)));
    TRY(check_workspace(workspace, workspace_bytes, need));
  }
  spans[10] = {dY, n * elem(y_dtype), false};
  spans[11] = {dX_out, n * elem(x_dtype), false};
  spans[12] = {X, n * elem(x_dtype), false};
  spans[13] = {H, n * elem(h_dtype), false};
  spans[14] = {dX, n * elem(x_dtype), true};
  spans[15] = {dH, n * elem(h_dtype), true};
  spans[16] = {workspace, need, true};
  TRY(check_spans(spans, 17));
  return svdq::launch_block_norm_grad(a, g, M, images, out, workspace, stream);
}

}  // extern "C"

// ------------------------------------------- AWQ product with an epilogue
namespace {

svdq_status check_act_or_none(svdq_act a) {
  if (a == SVDQ_NO_ACT) return SVDQ_OK;
  return check_act(a);
}

svdq_status check_images(int64_t M, int64_t images) {
  if (images <= 0 || images > MAX_IMAGES || M % images != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "images must be in [1, 2^20] and divide M");
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t awq_linear_w4a16_res_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_mkn(M, K, N) != SVDQ_OK) return 0;
  return svdq::awq_res_workspace(M, K, N);
}

svdq_status awq_linear_w4a16_res(const uint16_t* X, int64_t M, int64_t K, int64_t N, int32_t group,
                                 const uint8_t* q, const uint16_t* scales, const uint16_t* zeros,
                                 const uint16_t* bias, svdq_act act, const svdq_vec* gate,
                                 int64_t images, const void* R, svdq_dtype r_dtype, void* Y,
                                 svdq_dtype y_dtype, uint16_t* Z_out, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_act_or_none(act));
  TRY(check_dtype(y_dtype, "y_dtype"));
  if (R) TRY(check_dtype(r_dtype, "r_dtype"));
  TRY(check_mkn(M, K, N));
  TRY(check_tiles(M, N));
  TRY(check_images(M, images));
  if (M == 0) return SVDQ_OK;
  const svdq::AwqWeight w{q, scales, zeros};
  Span spans[10];
  svdq::ResEpilogue e{bias, {}, int(M / images), 0, R, r_dtype == SVDQ_BF16,
                      Y, y_dtype == SVDQ_BF16, Z_out};
  TRY(take_vec(gate, "gate", N, images, e.gate, spans[0]));
  TRY(check_ptr(X, "X"));
  TRY(check_awq(w, ""));
  if (bias) TRY(check_ptr(bias, "bias", 2));
  if (R) TRY(check_ptr(R, "R"));
  TRY(check_ptr(Y, "Y"));
  if (Z_out) TRY(check_ptr(Z_out, "Z_out"));
  const size_t need = svdq::awq_res_workspace(M, K, N);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t m = M, k = K, n = N;
  spans[1] = {X, m * k * 2, false};
  spans[2] = {q, n * k / 2, false};
  spans[3] = {scales, n * k / 32, false};
  spans[4] = {zeros, n * k / 32, false};
  spans[5] = {bias, n * 2, false};
  spans[6] = {R, m * n * elem(r_dtype), false};
  spans[7] = {Y, m * n * elem(y_dtype), true};
  spans[8] = {Z_out, m * n * 2, true};
  spans[9] = {workspace, need, true};
  TRY(check_spans(spans, 10));
  return svdq::launch_awq_res(X, M, K, N, w, act, e, workspace, stream);
}

size_t awq_linear_w4a16_res_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t images) {
  if (check_mkn(M, K, N) != SVDQ_OK || check_images(M, images) != SVDQ_OK) return 0;
  return svdq::awq_res_grad_workspace(M, K, N, images);
}

svdq_status awq_linear_w4a16_res_grad(const void* dY, svdq_dtype dy_dtype, const uint16_t* Z,
                                      int64_t M, int64_t K, int64_t N, int32_t group,
                                      const uint8_t* q, const uint16_t* scales,
                                      const uint16_t* zeros, svdq_act act, const svdq_vec* gate,
                                      int64_t images, uint16_t* dX, uint16_t* dZ, float* dgate,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_act_or_none(act));
  TRY(check_dtype(dy_dtype, "dy_dtype"));
  TRY(check_mkn(M, K, N));
  TRY(check_tiles(M, K));
  TRY(check_images(M, images));
  const svdq::AwqWeight w{q, scales, zeros};
  Span spans[10];
  svdq::Vec g;
  TRY(take_vec(gate, "gate", N, images, g, spans[0]));
  if (dgate) {
    if (!gate) return fail(SVDQ_ERR_INVALID_ARG, "dgate is asked for without gate");
    TRY(check_ptr(dgate, "dgate"));
  }
  const size_t m = M, k = K, n = N, need = M ? svdq::awq_res_grad_workspace(M, K, N, images) : 0;
  if (M) {
    TRY(check_ptr(dY, "dY"));
    if (Z || act != SVDQ_NO_ACT || dgate) TRY(check_ptr(Z, "Z"));
    TRY(check_awq(w, ""));
    TRY(check_ptr(dX, "dX"));
    TRY(check_ptr(dZ, "dZ"));
    TRY(check_workspace(workspace, workspace_bytes, need));
  }
  spans[1] = {dY, m * n * elem(dy_dtype), false};
  spans[2] = {Z, m * n * 2, false};
  spans[3] = {q, n * k / 2, false};
  spans[4] = {scales, n * k / 32, false};
  spans[5] = {zeros, n * k / 32, false};
  spans[6] = {dX, m * k * 2, true};
  spans[7] = {dZ, m * n * 2, true};
  spans[8] = {dgate, size_t(g.ld ? images : 1) * n * 4, true};
  spans[9] = {workspace, need, true};
  TRY(check_spans(spans, 10));
  return svdq::launch_awq_res_grad(dY, dy_dtype == SVDQ_BF16, Z, M, K, N, images, w, act, g, dX, dZ,
                                   dgate, workspace, stream);
}

}  // extern "C"

// ------------------------------------------------- mixture of experts
namespace {

svdq_status check_moe(int64_t T, int64_t E, int32_t top, int64_t K, int64_t N) {
  TRY(check_mkn(T, K, N));
  if (N % 64 != 0) return fail(SVDQ_ERR_INVALID_ARG, "N must be a positive multiple of 64");
  if (T > 64) return fail(SVDQ_ERR_UNSUPPORTED, "awq_moe_w4a16 takes at most 64 tokens");
  if (E <= 0) return fail(SVDQ_ERR_INVALID_ARG, "E must be positive");
  if (E > 256) return fail(SVDQ_ERR_UNSUPPORTED, "E must be at most 256");
  if (top <= 0 || top > E) return fail(SVDQ_ERR_INVALID_ARG, "top must be in [1, E]");
  if (top > 16) return fail(SVDQ_ERR_UNSUPPORTED, "top must be at most 16");
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t awq_moe_w4a16_workspace_bytes(int64_t T, int64_t E, int32_t top, int64_t K, int64_t N) {
  if (check_moe(T, E, top, K, N) != SVDQ_OK) return 0;
  return svdq::awq_moe_workspace(T, E, top, K, N);
}

svdq_status awq_moe_w4a16(const uint16_t* X, const void* logits, svdq_dtype logits_dtype, int64_t T,
                          int64_t E, int32_t top, int64_t K, int64_t N, int32_t group,
                          const uint8_t* q_gate, const uint16_t* scales_gate,
                          const uint16_t* zeros_gate, const uint8_t* q_up,
                          const uint16_t* scales_up, const uint16_t* zeros_up,
                          const uint8_t* q_down, const uint16_t* scales_down,
                          const uint16_t* zeros_down, svdq_act act, int32_t renorm, uint16_t* Y,
                          int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  svdq::clear_error();
  TRY(check_group(group));
  TRY(check_act(act));
  TRY(check_dtype(logits_dtype, "logits_dtype"));
  TRY(check_moe(T, E, top, K, N));
  if (T == 0) return SVDQ_OK;
  const svdq::AwqWeight g{q_gate, scales_gate, zeros_gate}, u{q_up, scales_up, zeros_up},
      d{q_down, scales_down, zeros_down};
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(logits, "logits", elem(logits_dtype)));
  TRY(check_awq(g, "_gate"));
  TRY(check_awq(u, "_up"));
  TRY(check_awq(d, "_down"));
  TRY(check_ptr(Y, "Y"));
  if (ids) TRY(check_ptr(ids, "ids", 4));
  if (weights) TRY(check_ptr(weights, "weights", 4));
  const size_t need = svdq::awq_moe_workspace(T, E, top, K, N);
  TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t t = T, e = E, k = K, n = N, c = size_t(T) * size_t(top) * 4;
  const Span spans[] = {{X, t * k * 2, false}, {logits, t * e * elem(logits_dtype), false},
                        {q_gate, e * n * k / 2, false}, {scales_gate, e * n * k / 32, false},
                        {zeros_gate, e * n * k / 32, false}, {q_up, e * n * k / 2, false},
                        {scales_up, e * n * k / 32, false}, {zeros_up, e * n * k / 32, false},
                        {q_down, e * n * k / 2, false}, {scales_down, e * n * k / 32, false},
                        {zeros_down, e * n * k / 32, false}, {Y, t * k * 2, true}, {ids, c, true},
                        {weights, c, true}, {workspace, need, true}};
  TRY(check_spans(spans, 15));
  return svdq::launch_awq_moe(X, logits, logits_dtype == SVDQ_BF16, T, E, top, K, N, g, u, d, act,
                              renorm != 0, Y, ids, weights, workspace, stream);
}

}  // extern "C"
