// The norm and residual operators around a block: what the C ABI hands on.
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
  int64_t D, rows;        // rows of one image
  float eps;
  Vec post, gate, weight, scale, shift;
};

struct BlockNormGrad {
  const void *dY, *dX_out;
  void *dX, *dH;
  bool y16;
  int64_t parts;          // workgroups an image
  float* part[5];         // partial sums of the vectors' gradients [workgroups][D]
};

svdq_status launch_block_norm(const BlockNorm& a, int64_t M, void* X_out, void* Y, svdq_dtype y_dt,
                              hipStream_t s);
size_t block_norm_grad_workspace(int64_t M, int64_t D, int64_t images);
// out: the gradients of post, gate, weight, scale and shift (NULL: not wanted), fp32
svdq_status launch_block_norm_grad(const BlockNorm& a, BlockNormGrad g, int64_t M, int64_t images,
                                   float* const (&out)[5], void* ws, hipStream_t s);

}  // namespace svdq
