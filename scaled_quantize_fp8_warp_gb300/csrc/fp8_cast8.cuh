// E4M3 bytes of eight consecutive elements under a fp32 scale, the cast of
// fp8_quantize_tile1x128 (s = max(amax / 448, 1e-12), RNE of the correctly
// rounded quotient x / s), as the activation-checkpoint and norm kernels use it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8_pack8.cuh"

namespace fp8q {
namespace tilecast {

using pack8::Pack8;

// A tile's scale from its max |x|.
__device__ __forceinline__ float tile_scale(uint32_t amax_bits) {
  const float s = __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
  return s < 1e-12f ? 1e-12f : s;
}

// E4M3 bytes of eight elements under a finite scale s with r = RN(1 / s):
// RN(x / s) by Markstein's correction.  Found as -q (q0 = x (-r), e = q0 s + x,
// q = e (-r) + q0), whose sign bits are turned at the end, so that a zero
// keeps x's sign.
template <typename T>
__device__ __forceinline__ uint2 cast8(const Pack8<T> &x, float s, float r) {
  uint32_t b[4];
  const float2 nr = make_float2(-r, -r), s2 = make_float2(s, s);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = x.pair(k), q = __fmul2_rn(v, nr);
    b[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(__ffma2_rn(__ffma2_rn(q, s2, v), nr, q),
                                              __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(__byte_perm(b[0], b[1], 0x5410) ^ 0x80808080u,
                    __byte_perm(b[2], b[3], 0x5410) ^ 0x80808080u);
}

// One element of a tile that is not finite: a NaN keeps its
// sign, a NaN that the division makes is 0x7F, and all else is a zero (s is
// infinite or NaN).
static __device__ __noinline__ uint32_t cast1_careful(float x, float s) {
  if (x != x) return 0x7Fu | ((__float_as_uint(x) >> 24) & 0x80u);
  const float q = __fdiv_rn(x, s);
  if (q != q) return 0x7Fu;
  return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

template <typename T>
__device__ __forceinline__ uint2 cast8_any(const Pack8<T> &x, float s, float r) {
  if (s < __uint_as_float(0x7F800000u)) return cast8(x, s, r);
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = cast1_careful(x.at(j), s);
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24),
                    b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}

template <bool VEC>
__device__ __forceinline__ void store_bytes(uint8_t *p, int valid, uint2 w) {
  if (VEC) {
    if (valid > 0) __stcs(reinterpret_cast<uint2 *>(p), w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) p[j] = (uint8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * (j - 4))) & 0xFFu);
}

}  // namespace tilecast
}  // namespace fp8q
