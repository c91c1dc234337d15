// Host-side declarations of the RMS norm kernels.
#pragma once

#include "fp8q_internal.h"

namespace fp8q {
namespace norm {

struct ForwardArgs {
  int64_t T, C;
  const void *x, *residual;    // residual: null where there is none (then h is too)
  int64_t ldx, ldr;
  const void *weight;
  int w_bf16;
  float eps;
  void *h, *y;                 // y: null where it is not wanted
  int64_t ldh, ldy;
  uint8_t *q;                  // [T, C] or null
  float *q_scales;             // [ceil(C/128), T], or [T] for row scaling
  int row_scale;
  float *rstd;                 // [T] or null
};

struct BackwardArgs {
  int64_t T, C;
  const void *dy, *h, *dresidual;   // dresidual: may be null
  int64_t lddy, ldh, lddr;
  const void *weight;
  int w_bf16;
  const float *rstd;
  void *dx;
  int64_t lddx;
  void *dweight;                    // [C] of the weight's type, or null
  float *partial;                   // [kPartials, C] where dweight is wanted
};

// Partial sums of dweight, one row of C for each CTA of the backward kernel:
// three CTAs at most on each of 152 SMs.
constexpr int kPartials = 3 * kNumSMsHint;

cudaError_t launch_forward(int dtype, const ForwardArgs &a, cudaStream_t stream);
cudaError_t launch_backward(int dtype, const BackwardArgs &a, cudaStream_t stream);

}  // namespace norm
}  // namespace fp8q
