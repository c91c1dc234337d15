// Activation functions with 8-bit checkpoints: a = f(u) or f(u) v forward,
// du = da f'(u) v and dv = da f(u) backward from E4M3 copies of u and v under
// 1x128 tile scales (the cast of fp8_quantize_tile1x128: s = max(amax / 448,
// 1e-12), RNE of the correctly rounded quotient x / s, reached by one
// reciprocal per tile and Markstein's correction).
//
// One warp owns 2 rows x 128 columns at a time: 16 lanes of 8 columns each a
// tile, whose maximum is a 4-step butterfly.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "fp8_act.h"

namespace fp8q {
namespace act {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// f(u), and f'(u) where it is wanted.  exp is the hardware's base-2
// exponential (about 2 units in the last place); large |u| stay finite: e^-u
// may overflow to infinity, whose reciprocal is 0.
template <int ACT, bool GRAD>
__device__ __forceinline__ void activation(float u, float &f, float &df) {
  if (ACT == FP8Q_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-u));
    f = u * s;
    if (GRAD) df = s * (1.0f + u * (1.0f - s));
  } else if (ACT == FP8Q_ACT_GELU) {
    const float p = 0.5f + 0.5f * erff(u * 0.70710678f);
    f = u * p;
    if (GRAD) df = p + u * (0.39894228f * __expf(-0.5f * u * u));
  } else {
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z)
    const float p = __fdividef(1.0f, 1.0f + __expf(-1.5957691f * u * (1.0f + 0.044715f * u * u)));
    f = u * p;
    if (GRAD) {
      const float q = p * (1.0f - p);
      df = p + (q == 0.0f ? 0.0f : u * q * 1.5957691f * (1.0f + 0.134145f * u * u));
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int valid, float (&v)[8]) {
  if (VEC && valid >= 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = *reinterpret_cast<const uint4 *>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4 *>(p);
      const float4 b = *(reinterpret_cast<const float4 *>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < valid ? (float)p[j] : 0.0f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int valid, const float (&v)[8]) {
  if (VEC && valid >= 8) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t *>(&b);
      }
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) p[j] = (T)v[j];
}

// One element where the tile is not finite: a NaN keeps its sign, a NaN that
// the division makes is 0x7F (s is infinite or NaN, so nothing else than
// zeros and NaN comes out).
__device__ __forceinline__ uint32_t cast1_slow(float x, float s) {
  if (x != x) return 0x7Fu | ((__float_as_uint(x) >> 24) & 0x80u);
  const float q = __fdiv_rn(x, s);
  if (q != q) return 0x7Fu;
  return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// The eight E4M3 bytes of this lane's part of a tile, and the tile's scale.
__device__ __forceinline__ uint2 cast_tile(const float (&v)[8], float &scale) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float q = __fdiv_rn(__uint_as_float(m), 448.0f);
  const float s = q < 1e-12f ? 1e-12f : q;
  scale = s;
  uint32_t b[8];
  if (m < 0x7F800000u) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 x = make_float2(v[j], v[j + 1]), r2 = make_float2(r, r);
      const float2 q0 = __fmul2_rn(x, r2);
      const float2 e = __ffma2_rn(q0, make_float2(-s, -s), x);
      float2 t = __ffma2_rn(e, r2, q0);
      t.x = copysignf(t.x, x.x);
      t.y = copysignf(t.y, x.y);
      b[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(b[0] | (b[2] << 16), b[4] | (b[6] << 16));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = cast1_slow(v[j], s);
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24),
                    b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}

template <bool VEC>
__device__ __forceinline__ void store_bytes(uint8_t *p, int valid, uint2 w) {
  if (VEC && valid >= 8) {
    *reinterpret_cast<uint2 *>(p) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) p[j] = (uint8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * (j - 4))) & 0xFFu);
}

// The values of this lane's eight bytes under scale s.
template <bool VEC>
__device__ __forceinline__ void load_saved(const uint8_t *p, int valid, float s, float (&v)[8]) {
  uint32_t w[2] = {0u, 0u};
  if (VEC && valid >= 8) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = t.x, w[1] = t.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = __fmul_rn(f.x, s);
    v[2 * j + 1] = __fmul_rn(f.y, s);
  }
}

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) forward_kernel(const ForwardArgs p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles = (p.F + 127) / 128, pairs = (p.T + 1) / 2;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + warp; n < tiles * pairs; n += step) {
    const int64_t pair = n / tiles, tile = n - pair * tiles;
    const int64_t row = 2 * pair + (lane >> 4), col = tile * 128 + (lane & 15) * 8;
    const int valid = row < p.T ? (int)max((int64_t)0, min((int64_t)8, p.F - col)) : 0;
    const int64_t at = valid > 0 ? 1 : 0;   // nothing is addressed where nothing is valid
    float u[8], v[8], a[8], s, unused;
    load8<T, VEC>(static_cast<const T *>(p.u) + at * (row * p.ldu + col), valid, u);
    if (GATED) load8<T, VEC>(static_cast<const T *>(p.v) + at * (row * p.ldv + col), valid, v);
    const uint2 bu = cast_tile(u, s);
    store_bytes<VEC>(p.u8 + at * (row * p.F + col), valid, bu);
    if ((lane & 15) == 0 && row < p.T) p.u_scales[tile * p.T + row] = s;
    if (GATED) {
      const uint2 bv = cast_tile(v, s);
      store_bytes<VEC>(p.v8 + at * (row * p.F + col), valid, bv);
      if ((lane & 15) == 0 && row < p.T) p.v_scales[tile * p.T + row] = s;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      activation<ACT, false>(u[j], a[j], unused);
      if (GATED) a[j] *= v[j];
    }
    store8<T, VEC>(static_cast<T *>(p.a) + at * (row * p.lda + col), valid, a);
  }
}

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BackwardArgs p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles = (p.F + 127) / 128, pairs = (p.T + 1) / 2;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + warp; n < tiles * pairs; n += step) {
    const int64_t pair = n / tiles, tile = n - pair * tiles;
    const int64_t row = 2 * pair + (lane >> 4), col = tile * 128 + (lane & 15) * 8;
    const int valid = row < p.T ? (int)max((int64_t)0, min((int64_t)8, p.F - col)) : 0;
    if (valid == 0) continue;
    float u[8], v[8], da[8], du[8], dv[8], a[8];
    load_saved<VEC>(p.u8 + row * p.F + col, valid, p.u_scales[tile * p.T + row], u);
    if (GATED) load_saved<VEC>(p.v8 + row * p.F + col, valid, p.v_scales[tile * p.T + row], v);
    load8<T, VEC>(static_cast<const T *>(p.da) + row * p.ldda + col, valid, da);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f, df;
      activation<ACT, true>(u[j], f, df);
      du[j] = GATED ? da[j] * v[j] * df : da[j] * df;
      dv[j] = da[j] * f;
      a[j] = GATED ? f * v[j] : f;
    }
    store8<T, VEC>(static_cast<T *>(p.du) + row * p.lddu + col, valid, du);
    if (GATED) store8<T, VEC>(static_cast<T *>(p.dv) + row * p.lddv + col, valid, dv);
    if (p.a != nullptr) store8<T, VEC>(static_cast<T *>(p.a) + row * p.lda + col, valid, a);
  }
}

int grid_for(int64_t T, int64_t F) {
  const int64_t warps = ((T + 1) / 2) * ((F + 127) / 128);
  return (int)std::min<int64_t>((warps + kThreads / 32 - 1) / (kThreads / 32), 8 * sm_count());
}

bool vec_ok(const void *p, int64_t ld, int64_t size) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0);
}

template <int ACT, typename T, bool GATED>
void forward(const ForwardArgs &a, bool vec, cudaStream_t stream) {
  const int grid = grid_for(a.T, a.F);
  if (vec)
    forward_kernel<ACT, T, GATED, true><<<grid, kThreads, 0, stream>>>(a);
  else
    forward_kernel<ACT, T, GATED, false><<<grid, kThreads, 0, stream>>>(a);
}

template <int ACT, typename T, bool GATED>
void backward(const BackwardArgs &a, bool vec, cudaStream_t stream) {
  const int grid = grid_for(a.T, a.F);
  if (vec)
    backward_kernel<ACT, T, GATED, true><<<grid, kThreads, 0, stream>>>(a);
  else
    backward_kernel<ACT, T, GATED, false><<<grid, kThreads, 0, stream>>>(a);
}

template <int ACT>
void forward_type(int dtype, const ForwardArgs &a, bool vec, cudaStream_t s) {
  const bool gated = a.v != nullptr;
  if (dtype == FP8Q_DT_BF16)
    gated ? forward<ACT, __nv_bfloat16, true>(a, vec, s) : forward<ACT, __nv_bfloat16, false>(a, vec, s);
  else
    gated ? forward<ACT, float, true>(a, vec, s) : forward<ACT, float, false>(a, vec, s);
}

template <int ACT>
void backward_type(int dtype, const BackwardArgs &a, bool vec, cudaStream_t s) {
  const bool gated = a.v8 != nullptr;
  if (dtype == FP8Q_DT_BF16)
    gated ? backward<ACT, __nv_bfloat16, true>(a, vec, s)
          : backward<ACT, __nv_bfloat16, false>(a, vec, s);
  else
    gated ? backward<ACT, float, true>(a, vec, s) : backward<ACT, float, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_forward(int act, int dtype, const ForwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.F % 16 == 0 && vec_ok(a.u, a.ldu, size) && vec_ok(a.v, a.ldv, size) &&
                   vec_ok(a.a, a.lda, size) && vec_ok(a.u8, a.F, 1) && vec_ok(a.v8, a.F, 1);
  if (act == FP8Q_ACT_SILU)
    forward_type<FP8Q_ACT_SILU>(dtype, a, vec, stream);
  else if (act == FP8Q_ACT_GELU)
    forward_type<FP8Q_ACT_GELU>(dtype, a, vec, stream);
  else
    forward_type<FP8Q_ACT_GELU_TANH>(dtype, a, vec, stream);
  return cudaGetLastError();
}

cudaError_t launch_backward(int act, int dtype, const BackwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.F % 16 == 0 && vec_ok(a.u8, a.F, 1) && vec_ok(a.v8, a.F, 1) &&
                   vec_ok(a.da, a.ldda, size) && vec_ok(a.du, a.lddu, size) &&
                   vec_ok(a.dv, a.lddv, size) && vec_ok(a.a, a.lda, size);
  if (act == FP8Q_ACT_SILU)
    backward_type<FP8Q_ACT_SILU>(dtype, a, vec, stream);
  else if (act == FP8Q_ACT_GELU)
    backward_type<FP8Q_ACT_GELU>(dtype, a, vec, stream);
  else
    backward_type<FP8Q_ACT_GELU_TANH>(dtype, a, vec, stream);
  return cudaGetLastError();
}

}  // namespace act
}  // namespace fp8q
