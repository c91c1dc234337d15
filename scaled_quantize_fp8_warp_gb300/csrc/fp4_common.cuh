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

// A block's scale byte and what dividing by the scale takes.
struct BlockScale {
  uint32_t byte;
  float d;   // NVFP4: the divisor; unused for MXFP4
  float r;   // MXFP4: 1 / d, exact; NVFP4: RN(1 / d); 0 where the block is not finite
  bool over; // NVFP4: the block's scale saturated, so quotients may pass 6 by any factor
};

template <int KIND>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, float g) {
  BlockScale b;
  const bool finite = amax_bits < 0x7F800000u;
  if (KIND == FP4Q_MXFP4) {
    // the biased exponent of amax is floor(log2 amax) + 127; zero, subnormal
    // and tiny maxima clamp to 2^-127
    const int e = (int)(amax_bits >> 23);
    b.byte = finite ? (uint32_t)max(e - 2, 0) : 0xFFu;
    b.d = 0.0f;
    b.over = false;
    // 2^(127 - byte), a normal number for every finite byte (at most 252)
    b.r = finite ? __uint_as_float((254u - b.byte) << 23) : 0.0f;
  } else {
    const float t = __fdiv_rn(__fdiv_rn(__uint_as_float(amax_bits), 6.0f), g);
    uint32_t s = (uint32_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    s = s == 0u ? 1u : s;                       // at least 2^-9
    const bool nan = !finite || !(t == t) || !(g < __uint_as_float(0x7F800000u));
    b.byte = nan ? 0x7Fu : s;
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s, __NV_E4M3);
    b.d = __fmul_rn(__half2float(__half(h)), g);
    b.r = nan ? 0.0f : __frcp_rn(b.d);
    b.over = t > 448.0f;
  }
  return b;
}

// Codes of two elements of a block (the first in the low four bits).
template <int KIND>
__device__ __forceinline__ uint32_t encode2(float lo, float hi, const BlockScale &b) {
  if (KIND == FP4Q_MXFP4) return e2m1x2(__fmul_rn(lo, b.r), __fmul_rn(hi, b.r));
  if (b.over) {   // keep the correction finite: everything past 6 d has the code of 6 d
    lo = fminf(fmaxf(lo, -6.5f * b.d), 6.5f * b.d);
    hi = fminf(fmaxf(hi, -6.5f * b.d), 6.5f * b.d);
  }
  const float2 x = make_float2(lo, hi), r = make_float2(b.r, b.r), nd = make_float2(-b.d, -b.d);
  const float2 q0 = __fmul2_rn(x, r);
  const float2 q = __ffma2_rn(__ffma2_rn(q0, nd, x), r, q0);
  return e2m1x2(copysignf(q.x, lo), copysignf(q.y, hi));   // a zero quotient keeps its sign
}

// Codes of eight elements, element j in bits [4j, 4j + 4).
template <int KIND>
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], const BlockScale &b) {
  const uint32_t w = encode2<KIND>(v[0], v[1], b) | (encode2<KIND>(v[2], v[3], b) << 8) |
                     (encode2<KIND>(v[4], v[5], b) << 16) | (encode2<KIND>(v[6], v[7], b) << 24);
  return b.r == 0.0f ? 0u : w;   // NaN or infinity in the block
}

// Value of one E2M1 code: exact in fp32.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp4_to_halfraw((__nv_fp4_storage_t)(code & 15u), __NV_E2M1);
  return __half2float(__half(h));
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
