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

// Up to kGroupMax matrices of one type, or products of one kind, in one launch.
constexpr int kGroupMax = 3;

// n non-empty matrices in one launch.
cudaError_t launch_quantize(int kind, int in_dtype, const QuantArgs *a, int n, cudaStream_t stream);
// amax[i] = max |x| of n dense matrices of size[i] elements, one launch.
cudaError_t launch_amax_group(const void *const *x, const int64_t *size, int n, int in_dtype,
                              float *amax, cudaStream_t stream);
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

// One product C[M,N] = A . B^T; A and B of one kind.
struct Product {
  fp4q_operand A, B;
  void *C;
  int64_t M, N, K;
};

// Whether a product's sizes fit the kernels' indexes: element offsets are
// 64-bit, but rows, tiles and scale atoms are counted in 32 bits, and the
// coordinates of a tile past the last row have to fit too.
bool product_fits(int kind, int64_t M, int64_t N, int64_t K);

// y[M,N] = x . w^T on tiles of 128 rows of w by up to 128 rows of x, K split
// over the CTAs of a cluster: n products in one launch, x their A.
int launch_split(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream);
// The same for one x in bf16 or fp32 that the kernel quantises as it goes (at
// most FP4Q_LINEAR_FUSED_ROWS rows; x_amax: NVFP4's amax); prod.A is unused.
int launch_split_quantizing(int kind, const void *x, int in_dtype, int64_t ldx,
                            const float *x_amax, const Product &prod, int out_dtype,
                            cudaStream_t stream);
// Microseconds beyond a launch's fixed cost that launch_split would take, by
// the model that chooses between it and CTA pairs.
double split_cost(int64_t M, int64_t N, int64_t K);

// n <= kGroupMax independent products that fit; a FP8Q status.
int launch_products(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream);

}  // namespace fp4
}  // namespace fp8q
