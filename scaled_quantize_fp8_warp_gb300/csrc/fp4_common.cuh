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

// NVFP4's 127 block scales of one tensor: d = fl32(s g) and RN(1 / d) by
// scale byte, so that no block needs a division of its own.
struct ScaleTable {
  float2 d_r[128];
  __device__ __forceinline__ void fill(float g) {   // by 128 threads or more, then a barrier
    if (threadIdx.x < 128) {
      const __half_raw h =
          __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)min(threadIdx.x, 126u), __NV_E4M3);
      const float d = __fmul_rn(__half2float(__half(h)), g);
      d_r[threadIdx.x] = make_float2(d, threadIdx.x == 0 ? 0.0f : __frcp_rn(d));
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

// A block's scale byte and what dividing by the scale takes.
struct BlockScale {
  uint32_t byte;
  float d;     // NVFP4: the divisor; unused for MXFP4
  float r;     // MXFP4: 1 / d, exact; NVFP4: RN(1 / d)
  bool nan;    // the block stands for NaN
  bool over;   // NVFP4: the scale saturated, so quotients may pass 6 by any factor
};

template <int KIND>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, float g, float rg,
                                                  const ScaleTable *table) {
  BlockScale b;
  b.nan = amax_bits >= 0x7F800000u;
  if (KIND == FP4Q_MXFP4) {
    // the biased exponent of amax is floor(log2 amax) + 127; zero, subnormal
    // and tiny maxima clamp to 2^-127, whose reciprocal is a normal number
    const uint32_t code = (uint32_t)max((int)(amax_bits >> 23) - 2, 0);
    b.byte = b.nan ? 0xFFu : code;
    b.d = 0.0f;
    b.r = __uint_as_float((254u - code) << 23);
    b.over = false;
  } else {
    const float t = nv_ratio(__uint_as_float(amax_bits), g, rg);
    uint32_t s = (uint32_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3) & 0x7Fu;
    s = min(max(s, 1u), 126u);                   // at least 2^-9
    b.nan = b.nan || !(g < __uint_as_float(0x7F800000u));
    b.byte = b.nan ? 0x7Fu : s;
    const float2 dr = table->d_r[s];
    b.d = dr.x;
    b.r = dr.y;
    b.over = t > 448.0f;
  }
  return b;
}

// Codes of two elements of a block, given negated (the first in the low four
// bits).  NVFP4: RN(x / d) by Markstein's correction, signs arranged so that a
// zero quotient keeps x's sign: q0 = x r, e = q0 d - x, q = q0 - e r.
template <int KIND>
__device__ __forceinline__ uint32_t encode2(float2 y, const BlockScale &b) {
  const float2 nr = make_float2(-b.r, -b.r);
  if (KIND == FP4Q_NVFP4 && b.over) {   // keep the correction finite: past 6 d the code is 6's
    const float lim = 6.5f * b.d;
    y.x = fminf(fmaxf(y.x, -lim), lim);
    y.y = fminf(fmaxf(y.y, -lim), lim);
  }
  float2 q = __fmul2_rn(y, nr);
  if (KIND == FP4Q_NVFP4) q = __ffma2_rn(__ffma2_rn(q, make_float2(b.d, b.d), y), nr, q);
  return e2m1x2(q.x, q.y);
}

// Codes of eight elements given as negated pairs, element j in bits
// [4j, 4j + 4).
template <int KIND>
__device__ __forceinline__ uint32_t encode8(float2 y0, float2 y1, float2 y2, float2 y3,
                                            const BlockScale &b) {
  const uint32_t lo = __byte_perm(encode2<KIND>(y0, b), encode2<KIND>(y1, b), 0x0040);
  const uint32_t hi = __byte_perm(encode2<KIND>(y2, b), encode2<KIND>(y3, b), 0x0040);
  return b.nan ? 0u : __byte_perm(lo, hi, 0x5410);
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
