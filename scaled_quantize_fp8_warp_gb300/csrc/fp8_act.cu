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
#include "fp8_pack8.cuh"

namespace fp8q {
namespace act {
namespace {

using pack8::Pack8;
using pack8::divide2;
using pack8::load;
using pack8::store;

constexpr int kThreads = 256;

// 2^x and 1 / x of the hardware, about 2 units in the last place; tiny results
// are zero, which no sum with 1 below notices.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// f(u), and f'(u) where it is wanted.  Large |u| stay finite: e^-u may
// overflow to infinity, whose reciprocal is 0.
template <int ACT, bool GRAD>
__device__ __forceinline__ void activation(float u, float &f, float &df) {
  if (ACT == FP8Q_ACT_SILU) {
    const float s = rcp_fast(1.0f + exp2_fast(-1.44269504f * u));
    f = u * s;
    if (GRAD) df = s * (1.0f + u * (1.0f - s));
  } else if (ACT == FP8Q_ACT_GELU) {
    const float p = 0.5f + 0.5f * erff(u * 0.70710678f);
    f = u * p;
    if (GRAD) df = p + u * (0.39894228f * exp2_fast(-0.72134752f * u * u));
  } else {
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z), 2 z log2(e) = u (2.302208 + 0.1029432 u^2)
    const float uu = u * u;
    const float p = rcp_fast(1.0f + exp2_fast(-u * (2.30220819f + 0.10294324f * uu)));
    f = u * p;
    if (GRAD) {
      const float q = p * (1.0f - p);
      df = p + (q == 0.0f ? 0.0f : u * q * (1.5957691f + 0.21406671f * uu));
    }
  }
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

// The eight E4M3 bytes of this lane's part of a tile whose max |x| is m, and
// the tile's scale.
template <typename T>
__device__ __forceinline__ uint2 cast_tile(const Pack8<T> &x, uint32_t m, float &scale) {
  const float q = __fdiv_rn(__uint_as_float(m), 448.0f);
  const float s = q < 1e-12f ? 1e-12f : q;
  scale = s;
  uint32_t b[8];
  if (m < 0x7F800000u) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      b[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(divide2(x.pair(k), s, r), __NV_SATFINITE,
                                                __NV_E4M3);
    return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = cast1_slow(x.at(j), s);
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

template <bool VEC>
__device__ __forceinline__ uint2 load_bytes(const uint8_t *p, int valid) {
  if (VEC && valid >= 8) return *reinterpret_cast<const uint2 *>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

// The values of eight bytes under scale s.
__device__ __forceinline__ void saved(uint2 w, float s, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = __fmul_rn(f.x, s);
    v[2 * j + 1] = __fmul_rn(f.y, s);
  }
}

// The pieces (2 rows x 128 columns) of a [T, F] matrix that one warp visits:
// numbered row pair after row pair, `step` apart, kept as (pair, tile)
// without a division per piece.
struct Walk {
  int64_t pair, pairs;
  int tile, tiles;
  int64_t step_pair;
  int step_tile;
  __device__ __forceinline__ Walk(int64_t T, int64_t F) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    tiles = (int)((F + 127) / 128);
    pairs = (T + 1) / 2;
    pair = first / tiles;
    tile = (int)(first - pair * tiles);
    step_pair = step / tiles;
    step_tile = (int)(step - step_pair * tiles);
  }
  __device__ __forceinline__ bool in() const { return pair < pairs; }
  __device__ __forceinline__ void next() {
    pair += step_pair;
    tile += step_tile;
    if (tile >= tiles) {
      tile -= tiles;
      ++pair;
    }
  }
};

// This lane's 8 elements of a piece: row, first column, how many exist.
struct Place {
  int64_t row;
  int64_t col;
  int tile, valid;
  __device__ __forceinline__ Place(const Walk &w, int64_t T, int64_t F) {
    const int lane = threadIdx.x & 31;
    row = 2 * w.pair + (lane >> 4);
    tile = w.tile;
    col = (int64_t)tile * 128 + (lane & 15) * 8;
    valid = w.in() && row < T ? (int)max((int64_t)0, min((int64_t)8, F - col)) : 0;
  }
};

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) forward_kernel(const ForwardArgs p) {
  const int lane = threadIdx.x & 31;
  Walk walk(p.T, p.F);
  while (walk.in()) {
    // two pieces at a time: their loads are in flight together
    Place at[2] = {Place(walk, p.T, p.F), (walk.next(), Place(walk, p.T, p.F))};
    walk.next();
    Pack8<T> u[2], v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // nothing is addressed where nothing is valid
      const int64_t on = at[i].valid > 0 ? 1 : 0;
      load<VEC>(u[i], static_cast<const T *>(p.u) + on * (at[i].row * p.ldu + at[i].col), at[i].valid);
      if (GATED)
        load<VEC>(v[i], static_cast<const T *>(p.v) + on * (at[i].row * p.ldv + at[i].col), at[i].valid);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Place &a = at[i];
      uint32_t mu = u[i].amax_bits(), mv = GATED ? v[i].amax_bits() : 0u;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        mu = max(mu, __shfl_xor_sync(0xFFFFFFFFu, mu, o));
        if (GATED) mv = max(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o));
      }
      float su, sv = 0.0f;
      const uint2 bu = cast_tile(u[i], mu, su);
      uint2 bv = make_uint2(0u, 0u);
      if (GATED) bv = cast_tile(v[i], mv, sv);
      if (a.valid > 0) {
        store_bytes<VEC>(p.u8 + a.row * p.F + a.col, a.valid, bu);
        if (GATED) store_bytes<VEC>(p.v8 + a.row * p.F + a.col, a.valid, bv);
        if ((lane & 15) == 0) {
          p.u_scales[a.tile * p.T + a.row] = su;
          if (GATED) p.v_scales[a.tile * p.T + a.row] = sv;
        }
        float out[8], unused;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          activation<ACT, false>(u[i].at(j), out[j], unused);
          if (GATED) out[j] *= v[i].at(j);
        }
        store<VEC>(static_cast<T *>(p.a) + a.row * p.lda + a.col, a.valid, out);
      }
    }
  }
}

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BackwardArgs p) {
  Walk walk(p.T, p.F);
  while (walk.in()) {
    Place at[2] = {Place(walk, p.T, p.F), (walk.next(), Place(walk, p.T, p.F))};
    walk.next();
    Pack8<T> d[2];
    uint2 bu[2], bv[2];
    float su[2], sv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Place &a = at[i];
      if (a.valid > 0) {
        bu[i] = load_bytes<VEC>(p.u8 + a.row * p.F + a.col, a.valid);
        su[i] = p.u_scales[a.tile * p.T + a.row];
        if (GATED) {
          bv[i] = load_bytes<VEC>(p.v8 + a.row * p.F + a.col, a.valid);
          sv[i] = p.v_scales[a.tile * p.T + a.row];
        }
        load<VEC>(d[i], static_cast<const T *>(p.da) + a.row * p.ldda + a.col, a.valid);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Place &a = at[i];
      if (a.valid == 0) continue;
      float u[8], v[8], du[8], dv[8], out[8];
      saved(bu[i], su[i], u);
      if (GATED) saved(bv[i], sv[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f, df;
        const float da = d[i].at(j);
        activation<ACT, true>(u[j], f, df);
        du[j] = GATED ? da * v[j] * df : da * df;
        dv[j] = da * f;
        out[j] = GATED ? f * v[j] : f;
      }
      store<VEC>(static_cast<T *>(p.du) + a.row * p.lddu + a.col, a.valid, du);
      if (GATED) store<VEC>(static_cast<T *>(p.dv) + a.row * p.lddv + a.col, a.valid, dv);
      if (p.a != nullptr) store<VEC>(static_cast<T *>(p.a) + a.row * p.lda + a.col, a.valid, out);
    }
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
