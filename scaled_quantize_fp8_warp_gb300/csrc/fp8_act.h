// Host-side declarations of the activation-checkpoint kernels.
#pragma once

#include "fp8q_internal.h"

namespace fp8q {
namespace act {

struct ForwardArgs {
  int64_t T, F;
  const void *u, *v;           // v: null for an ungated activation
  int64_t ldu, ldv;
  void *a;
  int64_t lda;
  uint8_t *u8, *v8;            // [T, F]
  float *u_scales, *v_scales;  // [ceil(F/128), T]
};

struct BackwardArgs {
  int64_t T, F;
  const uint8_t *u8, *v8;
  const float *u_scales, *v_scales;
  const void *da;
  void *du, *dv, *a;           // a: null where it is not wanted
  int64_t ldda, lddu, lddv, lda;
};

cudaError_t launch_forward(int act, int dtype, const ForwardArgs &a, cudaStream_t stream);
cudaError_t launch_backward(int act, int dtype, const BackwardArgs &a, cudaStream_t stream);

}  // namespace act
}  // namespace fp8q
