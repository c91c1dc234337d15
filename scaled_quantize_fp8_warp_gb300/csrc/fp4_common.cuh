// Device-side definitions of the 4-bit formats: E2M1 codes, the E8M0 scale of
// an MXFP4 block and the E4M3 x fp32 scale of an NVFP4 block.
//
// E2M1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign.  All of a block's
// elements are divided by the block's scale d and rounded to nearest even,
// saturating at 6:
//   MXFP4 (OCP Microscaling Formats v1.0): 32 elements, d = 2^(code - 127)
//     with code - 127 = floor(log2 amax) - 2 (6 = 1.5 * 2^2).  d is a power
//     of two, so the quotient is an exact product.
//   NVFP4: 16 elements, d = fl32(s g) with g = max(fl32(amax / 2688), 1e-12)
//     for the whole tensor (2688 = 6 * 448) and s the block's E4M3 scale,
//     RNE(fl32(fl32(block amax / 6) / g)) within [2^-9, 448].  The floor of
//     2^-9, E4M3's smallest magnitude, keeps a block far below the tensor's
//     amax from dividing by zero.  The quotient is the correctly rounded fp32
//     division, reached as elsewhere in this library by one reciprocal per
//     block and Markstein's correction (P. Markstein, IBM J. Res. Dev. 34(1),
//     1990), whose remainder can only underflow where the code is zero.
// A block that holds a NaN or an infinity gets the scale's NaN code and zero
// elements: it stands for NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fp8q.h"

namespace fp8q {
namespace fp4 {

template <int KIND>
struct Kind;
template <>
struct Kind<FP4Q_MXFP4> {
  static constexpr int kBlock = 32;     // elements per scale
  static constexpr int kAtomK = 128;    // K that one 512-byte scale atom covers
};
template <>
struct Kind<FP4Q_NVFP4> {
  static constexpr int kBlock = 16;
  static constexpr int kAtomK = 64;
};

// E2M1 codes of two values, the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

// The tensor scale of NVFP4.  A NaN amax gives a NaN scale.
__device__ __forceinline__ float nv_global(float amax) {
  const float g = __fdiv_rn(amax, 2688.0f);
  return g < 1e-12f ? 1e-12f : g;
}

// NVFP4's 126 block scales of one tensor: d = fl32(s g) and RN(1 / d) by
// scale byte, so that no block needs a division of its own.
struct ScaleTable {
  float2 d_r[128];
  __device__ __forceinline__ void fill(float g) {   // by 128 threads or more, then a barrier
    if (threadIdx.x < 128) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(
          (__nv_fp8_storage_t)min(max(threadIdx.x, 1u), 126u), __NV_E4M3);
      const float d = __fmul_rn(__half2float(__half(h)), g);
      d_r[threadIdx.x] = make_float2(d, __frcp_rn(d));
    }
  }
};

// RN(RN(amax / 6) / g) with rg = RN(1 / g), each quotient by Markstein's
// correction.  Past 512 the scale saturates, below 2^-10 it is the smallest:
// there the quotient need not be exact (and the correction may overflow).
__device__ __forceinline__ float nv_ratio(float amax, float g, float rg) {
  const float r6 = 1.0f / 6.0f;
  const float a0 = __fmul_rn(amax, r6);
  const float a = __fmaf_rn(__fmaf_rn(a0, -6.0f, amax), r6, a0);
  const float t0 = __fmul_rn(a, rg);
  return t0 > 512.0f ? t0 : __fmaf_rn(__fmaf_rn(t0, -g, a), rg, t0);
}

// Block maxima from here on take the careful path: NaN and infinity, and
// magnitudes so large that x / d may overflow where a calibrated amax is far
// too small (d >= 448e-12 > 2^-32 wherever the quotient is past 6).
constexpr uint32_t kCarefulBits = 0x6F800000u;   // 2^96

// -q for two elements of a block, q the quotient by its d; r = RN(1 / d).
// MXFP4: d is a power of two and the product exact.  NVFP4: RN(x / d) by
// Markstein's correction; as -q (q0 = x (-r), e = q0 d + x, e (-r) + q0), because
// a zero quotient then has the sign opposite to x's whatever that is.
template <int KIND>
__device__ __forceinline__ uint32_t encode2(float2 x, float d, float r) {
  const float2 nr = make_float2(-r, -r);
  float2 q = __fmul2_rn(x, nr);
  if (KIND == FP4Q_NVFP4) q = __ffma2_rn(__ffma2_rn(q, make_float2(d, d), x), nr, q);
  return e2m1x2(q.x, q.y);
}

// Codes of eight elements, element j in bits [4j, 4j + 4); the signs turn here.
template <int KIND>
__device__ __forceinline__ uint32_t encode8(const float2 (&x)[4], float d, float r) {
  const uint32_t lo = __byte_perm(encode2<KIND>(x[0], d, r), encode2<KIND>(x[1], d, r), 0x0040);
  const uint32_t hi = __byte_perm(encode2<KIND>(x[2], d, r), encode2<KIND>(x[3], d, r), 0x0040);
  return __byte_perm(lo, hi, 0x5410) ^ 0x88888888u;
}

// 1 / d of an MXFP4 block by scale byte: d = 2^(byte - 127) and the byte is
// at most 252, so the reciprocal is a normal number.
__device__ __forceinline__ float mx_reciprocal(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Scale byte of a block with a finite maximum below 2^96.
__device__ __forceinline__ uint32_t mx_byte(uint32_t amax_bits) {
  // the biased exponent of amax is floor(log2 amax) + 127; zero, subnormal
  // and tiny maxima clamp to 2^-127
  return (uint32_t)max((int)(amax_bits >> 23) - 2, 0);
}

// The careful path: scale byte and codes of eight elements for any maximum
// and any tensor scale.
template <int KIND>
__device__ __noinline__ uint32_t encode8_careful(float2 x0, float2 x1, float2 x2, float2 x3,
                                                 uint32_t amax_bits, float g, uint32_t *byte) {
  bool nan = amax_bits >= 0x7F800000u;
  float2 x[4] = {x0, x1, x2, x3};
  float d = 0.0f, r;
  if (KIND == FP4Q_MXFP4) {
    *byte = nan ? 0xFFu : mx_byte(amax_bits);
    r = nan ? 0.0f : mx_reciprocal(*byte);
  } else {
    nan = nan || !(g < __uint_as_float(0x7F800000u));
    const float t = __fdiv_rn(__fdiv_rn(__uint_as_float(amax_bits), 6.0f), g);
    const uint32_t s =
        (uint32_t)__nv_cvt_float_to_fp8(fmaxf(t, 0x1p-9f), __NV_SATFINITE, __NV_E4M3);
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s, __NV_E4M3);
    *byte = nan ? 0x7Fu : s;
    d = __fmul_rn(__half2float(__half(h)), g);
    r = __frcp_rn(d);
    const float lim = 6.5f * d;   // past 6 d the code is 6's
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = make_float2(fminf(fmaxf(x[k].x, -lim), lim), fminf(fmaxf(x[k].y, -lim), lim));
  }
  return nan ? 0u : encode8<KIND>(x, d, r);
}

// Values of the two codes in a byte, the low one first: exact in fp32.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(byte & 0xFFu), __NV_E2M1);
  return __half22float2(__half2(h));
}

// Value of a scale byte.
template <int KIND>
__device__ __forceinline__ float scale_value(uint32_t byte, float g) {
  if (KIND == FP4Q_MXFP4) {
    if (byte == 0xFFu) return __uint_as_float(0x7FFFFFFFu);
    return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
  }
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __fmul_rn(__half2float(__half(h)), g);
}

// Bytes of one row of codes, and the byte of scale (row, block) in the atoms.
__host__ __device__ inline int64_t row_bytes(int64_t K) { return (K + 31) / 32 * 16; }
__host__ __device__ inline int64_t num_atoms_k(int kind, int64_t K) {
  return kind == FP4Q_MXFP4 ? (K + 127) / 128 : (K + 63) / 64;
}
__host__ __device__ inline int64_t atom_byte(int64_t row, int64_t block, int64_t atoms_k) {
  return ((row >> 7) * atoms_k + (block >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 +
         (block & 3);
}

}  // namespace fp4
}  // namespace fp8q
