// Host-side declarations shared by the 4-bit and activation-checkpoint files.
#pragma once

#include "fp8q_internal.h"

namespace fp8q {
namespace fp4 {

struct QuantArgs {
  const void *x;
  int64_t rows, cols, ld;      // x: element (r, c) at r * ld + c
  const float *amax;           // NVFP4: device max |x|
  uint8_t *q, *q_scales;       // [rows, row_bytes(cols)] and its atoms, or null
  uint8_t *qt, *qt_scales;     // [cols, row_bytes(rows)] and its atoms, or null
  float *global_scale;         // NVFP4: receives g, or null
};

cudaError_t launch_quantize(int kind, int in_dtype, const QuantArgs &a, cudaStream_t stream);
// *global_scale = the tensor scale of *amax.
cudaError_t launch_global(const float *amax, float *global_scale, cudaStream_t stream);
// max |x| of a matrix with rows ld elements apart; *amax is zeroed first.
cudaError_t launch_amax_ld(const void *x, int in_dtype, int64_t rows, int64_t cols, int64_t ld,
                           float *amax, cudaStream_t stream);
cudaError_t launch_dequantize(int kind, const fp4q_operand &op, int64_t rows, int64_t K,
                              int out_dtype, void *y, cudaStream_t stream);

// Tensor maps of an operand's codes (box: 128 bytes of K x box_rows, 128-byte
// swizzle) and of its scale atoms as rows of 128 words (box: that many atoms).
bool make_tmap(CUtensorMap *m, const void *base, int64_t rows, int64_t K, uint32_t box_rows);
bool make_scale_tmap(CUtensorMap *m, const uint8_t *scales, int64_t rows, int64_t atoms_k,
                     uint32_t box);

// y[M,N] = x . w^T on tiles of 128 rows of w by up to 128 rows of x, K split
// over the CTAs of a cluster.  x is either the 4-bit operand `q` or, with q
// null, a bf16 / fp32 matrix that the kernel quantises as it goes (M at most
// FP4Q_LINEAR_FUSED_ROWS; x_amax: NVFP4's amax).
// Microseconds beyond a launch's fixed cost that launch_split would take for a
// quantised x, by the model that chooses between it and CTA pairs.
double split_cost(int64_t M, int64_t N, int64_t K);
int launch_split(int kind, const void *x, int in_dtype, int64_t ldx, const float *x_amax,
                 const fp4q_operand *q, const fp4q_operand &w, int out_dtype, void *y, int64_t M,
                 int64_t N, int64_t K, cudaStream_t stream);

// C[M,N] = A . B^T for non-empty sizes; a FP8Q status.
int launch_gemm(int kind, const fp4q_operand &A, const fp4q_operand &B, int out_dtype, void *C,
                int64_t M, int64_t N, int64_t K, cudaStream_t stream);

}  // namespace fp4
}  // namespace fp8q
