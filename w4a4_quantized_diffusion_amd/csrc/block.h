// The operators around a block's layers (norms, residual sums, epilogues): what the C
// ABI hands on.
#pragma once

#include "w4a16.h"

namespace svdq {

// a vector of D per image (ld elements apart) or for all rows (ld 0); p NULL: absent
struct Vec {
  const void* p;
  int64_t ld;
  bool b16;
};

struct BlockNorm {
  const void *X, *H;      // [M, D]; H may be NULL
  bool x16, h16, layer;
  int64_t D, images, rows;  // rows of one image
  float eps;
  double per;             // 1 / D
  Vec post, gate, weight, scale, shift;
};

struct BlockNormGrad {
  const void *dY, *dX_out;
  void *dX, *dH;
  bool y16;
  int64_t parts;          // workgroups an image
  float* grad[5];         // gradients of vectors that are one workgroup's sums [workgroups][D]
  float* sums[3];         // the workgroups' A, B and S [workgroups][D], for the others
};

// Sums of partial results, up to five in one launch: to[i][D] = the sum over the parts of
// image i (`parts` an image) of from [images parts][D], or the sum over all of them where
// `each` is 1, times the image's factor vector + add (1 if there is none).  In a fixed
// order; zeros for no parts.
struct Joins {
  int count;
  int64_t parts, images;
  const float* from[5];
  float* to[5];
  Vec factor[5];
  float plus[5];
  int64_t each[5];

  void add(const float* f, float* t, int64_t e, const Vec& v = {nullptr, 0, false}, float p = 0.f) {
    from[count] = f;
    to[count] = t;
    each[count] = e;
    factor[count] = v;
    plus[count++] = p;
  }
};
svdq_status launch_joins(const Joins& j, int64_t D, hipStream_t s);

// Epilogue of an AWQ product: Y = R + gate * act(Z), Z = the product + bias
struct ResEpilogue {
  const uint16_t* bias;   // [N] or NULL
  Vec gate;
  int rows, first;        // rows of one image; the image rows before the call's first row
  const void* R;          // [M, N] or NULL
  bool r16;
  void* Y;
  bool y16;
  uint16_t* Z;            // [M, N] or NULL
};
size_t awq_res_workspace(int64_t M, int64_t K, int64_t N);
svdq_status launch_awq_res(const uint16_t* X, int64_t M, int64_t K, int64_t N, AwqWeight w,
                           svdq_act act, const ResEpilogue& e, void* ws, hipStream_t s);
size_t awq_res_grad_workspace(int64_t M, int64_t K, int64_t N, int64_t images);
svdq_status launch_awq_res_grad(const void* dY, bool dy16, const uint16_t* Z, int64_t M, int64_t K,
                                int64_t N, int64_t images, AwqWeight w, svdq_act act, Vec gate,
                                uint16_t* dX, uint16_t* dZ, float* dgate, void* ws, hipStream_t s);

// dX = dZ wd in bf16, as launch_awq_linear_grad, with a last round of tiles split where
// that is faster (awq_grad.hip)
size_t awq_grad_product_workspace(int64_t M, int64_t K, int64_t N);
svdq_status launch_awq_grad_product(const uint16_t* dZ, int64_t M, int64_t K, int64_t N, AwqWeight w,
                                    uint16_t* dX, void* ws, hipStream_t s);

// At most 64 rows without dgate: dZ and dX in the product's own launches (awq_grad.hip),
// workspace as awq_linear_grad_workspace
bool awq_res_grad_fused(int64_t M, int64_t K, int64_t N);
svdq_status launch_awq_res_grad_rows(const uint16_t* dY, const uint16_t* Z, int64_t M, int64_t K,
                                     int64_t N, int64_t images, AwqWeight w, svdq_act act, Vec gate,
                                     uint16_t* dX, uint16_t* dZ, void* ws, hipStream_t s);

// Mixture of experts on AWQ weights, expert after expert (every one K N / 64 rows of 32
// bytes of codes)
size_t awq_moe_workspace(int64_t T, int64_t E, int64_t top, int64_t K, int64_t N);
svdq_status launch_awq_moe(const uint16_t* X, const void* logits, bool l16, int64_t T, int64_t E,
                           int64_t top, int64_t K, int64_t N, AwqWeight gate, AwqWeight up,
                           AwqWeight down, svdq_act act, bool renorm, uint16_t* Y, int32_t* ids,
                           float* weights, void* ws, hipStream_t s);

svdq_status launch_block_norm(const BlockNorm& a, int64_t M, void* X_out, void* Y, svdq_dtype y_dt,
                              hipStream_t s);
size_t block_norm_grad_workspace(int64_t M, int64_t D, int64_t images);
// out: the gradients of post, gate, weight, scale and shift (NULL: not wanted), fp32
svdq_status launch_block_norm_grad(const BlockNorm& a, BlockNormGrad g, int64_t M, int64_t images,
                                   float* const (&out)[5], void* ws, hipStream_t s);

}  // namespace svdq
