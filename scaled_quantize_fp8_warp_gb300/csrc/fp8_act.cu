// Activation functions with 8-bit checkpoints: a = f(u) or f(u) v forward,
// du = da f'(u) v and dv = da f(u) backward from E4M3 copies of u and v under
// 1x128 tile scales (the cast of fp8_quantize_tile1x128: s = max(amax / 448,
// 1e-12), RNE of the correctly rounded quotient x / s, reached by one
// reciprocal per tile and Markstein's correction).
//
// A warp works on 2 rows x 256 columns at a time: two tiles of each row, 16
// lanes of 8 columns to a tile.
//
// What bounds it: HBM.  Forward, gated SiLU bf16, 8.06 bytes an element: 15872 x
// 16384 326 us (6.4 TB/s, 95% of a copy's rate), 4096 x 8192 46 us (5.9); with
// three CTAs an SM 358 and 50.  Backward with the activation again, 10.06 bytes:
// 8192 x 16384 209 us (6.5 TB/s), 15872 x 4096 103 us (6.3).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp8_act.h"
#include "fp8_cast8.cuh"
#include "fp8_pack8.cuh"

namespace fp8q {
namespace act {
namespace {

using tilecast::cast8;
using tilecast::cast8_any;
using tilecast::store_bytes;
using tilecast::tile_scale;
using pack8::Pack8;
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

// The normal distribution below -v, v >= 0, from e = e^(-v^2/2): e t P(t) with
// t = 1 / (1 + v / sqrt 8), the form of C. Hastings (Approximations for Digital
// Computers, 1955).  P, of degree 8, was fitted for this file to erfcx(v / sqrt
// 2) / (2 t) with least largest relative error (4.3e-8 for v up to 13.5, where e
// underflows; 3.2e-7 in fp32).  (1 + erf) / 2 instead would lose every digit
// below -5.5; erfcf took 299 us where this takes 180 and erff took 206 (forward,
// gated bf16 8192 x 16384).
__device__ __forceinline__ float normal_tail(float v, float e) {
  const float t = rcp_fast(fmaf(v, 0.353553391f, 1.0f));
  float q = fmaf(t, -0.0294656865f, 0.141950533f);
  q = fmaf(t, q, -0.242899209f);
  q = fmaf(t, q, 0.13822794f);
  q = fmaf(t, q, -0.0127546927f);
  q = fmaf(t, q, 0.101105742f);
  q = fmaf(t, q, 0.121612407f);
  q = fmaf(t, q, 0.141179264f);
  q = fmaf(t, q, 0.141043693f);
  return q * (t * e);
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
    const float e = exp2_fast(-0.72134752f * u * u), q = normal_tail(fabsf(u), e);
    const float p = u < 0.0f ? q : 1.0f - q;
    f = u * p;
    if (GRAD) df = p + u * (0.39894228f * e);
  } else {
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z), 2 z log2(e) = u (2.302208 + 0.1029432 u^2)
    const float uu = u * u;
    const float p = rcp_fast(1.0f + exp2_fast(-u * (2.30220819f + 0.10294324f * uu)));
    f = u * p;
    if (GRAD) {
      const float q = p * (1.0f - p);
      df = p + (q == 0.0f ? 0.0f : u * q * (1.5957691f + 0.21406445f * uu));
    }
  }
}

template <bool VEC>
__device__ __forceinline__ uint2 load_bytes(const uint8_t *p, int valid) {
  if (VEC) return *reinterpret_cast<const uint2 *>(p);
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

// One warp keeps to one strip of two tile columns (256 columns) and walks down
// row pairs of it, with pointers that advance by constants; the second tile
// lies at constant offsets from the first.  Lanes 0-15 have a pair's first row.
// BLOCKED: consecutive pairs, so that a warp's scales are neighbours (the
// forward pass); otherwise the strip's warps take turns (the backward pass: 4%
// faster at 15872 x 4096, 1% at 8192 x 16384).
template <bool BLOCKED>
struct Walk {
  int strip, strip_step, strips;   // strips this warp serves
  int pair0, pairs, step;          // and row pairs pair0, pair0 + step, ... < pairs of each
  __device__ __forceinline__ Walk(int64_t T, int64_t F) {
    const int w = (int)blockIdx.x * (kThreads / 32) + (int)(threadIdx.x >> 5);
    const int all = (int)gridDim.x * (kThreads / 32);
    strips = (int)((F + 255) / 256);
    const int total = (int)((T + 1) / 2), share = max(all / strips, 1);   // warps per strip
    const int per = (total + share - 1) / share, mine = w / strips;
    strip_step = all < strips ? all : strips;
    strip = mine < share ? w - mine * strips : strips;   // the warps left over have none
    pair0 = BLOCKED ? mine * per : mine;
    pairs = BLOCKED ? min(total, pair0 + per) : total;
    step = BLOCKED ? 1 : share;
  }
};

// This lane's columns in a strip: the first of its eight in the first tile
// (those in the second are 128 further on), and how many of each exist.
struct Columns {
  int64_t col;
  int in[2];
  __device__ __forceinline__ Columns(int strip, int64_t F) {
    col = (int64_t)strip * 256 + (threadIdx.x & 15) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      in[i] = (int)max((int64_t)0, min((int64_t)8, F - (col + 128 * i)));
    if (in[0] == 0) col = 0;   // nothing is addressed where nothing is valid
  }
};

// Scales and reciprocals of the four tiles (two of u, two of v) of a half warp
// from the lanes' maxima: the halving steps leave tile 0's maxima in even
// lanes and tile 1's in odd ones, each lane finds one tile's scale (lane bit
// 1: u or v), and the results are handed round.
struct Scales {
  float s[2][2], r[2][2];   // [tile][u, v]
  bool finite;              // all four of every half warp
};

__device__ __forceinline__ void finish_scales(uint32_t mine, Scales &out) {
  const int lane = threadIdx.x & 31;
  out.finite = __all_sync(0xFFFFFFFFu, mine < 0x7F800000u);
  // RN(m / 448) by Markstein's correction, exact where it is not below 1e-12
  const float m = __uint_as_float(mine), c = 1.0f / 448.0f, q = __fmul_rn(m, c);
  float s = __fmaf_rn(__fmaf_rn(q, -448.0f, m), c, q);
  s = s < 1e-12f ? 1e-12f : s;
  if (!out.finite) s = tile_scale(mine);
  const float r = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int from = (lane & 16) + i + 2 * k;
      out.s[i][k] = __shfl_sync(0xFFFFFFFFu, s, from);
      out.r[i][k] = __shfl_sync(0xFFFFFFFFu, r, from);
    }
}

template <bool GATED>
__device__ __forceinline__ void find_scales(const Pack8<__nv_bfloat16> (&u)[2],
                                            const Pack8<__nv_bfloat16> (&v)[2], Scales &out) {
  const int lane = threadIdx.x & 31;
  // magnitudes of u in the low and of v in the high half
  uint32_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m[i] = __byte_perm(u[i].amax_bits(), GATED ? v[i].amax_bits() : 0u, 0x7632);
  const bool odd = lane & 1;
  uint32_t t = __vmaxu2(odd ? m[1] : m[0], __shfl_xor_sync(0xFFFFFFFFu, odd ? m[0] : m[1], 1));
#pragma unroll
  for (int o = 2; o < 16; o <<= 1) t = __vmaxu2(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  finish_scales((lane & 2) ? t & 0xFFFF0000u : t << 16, out);
}

template <bool GATED>
__device__ __forceinline__ void find_scales(const Pack8<float> (&u)[2], const Pack8<float> (&v)[2],
                                            Scales &out) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, two = lane & 2;
  uint32_t m[2];   // u, v of this lane's tile
#pragma unroll
  for (int k = 0; k < (GATED ? 2 : 1); ++k) {
    const uint32_t a = k ? v[0].amax_bits() : u[0].amax_bits();
    const uint32_t b = k ? v[1].amax_bits() : u[1].amax_bits();
    m[k] = max(odd ? b : a, __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1));
  }
  uint32_t t = m[0];
  if (GATED) t = max(two ? m[1] : m[0], __shfl_xor_sync(0xFFFFFFFFu, two ? m[0] : m[1], 2));
  else t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
#pragma unroll
  for (int o = 4; o < 16; o <<= 1) t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  finish_scales(t, out);
}

// Each thread keeps kStages steps' inputs (two tiles of one row) in shared
// memory slots of its own, filled by asynchronous copies a step ahead (VEC)
// -- no thread reads another's, so no barrier is needed.
constexpr int kStages = 2;

struct __align__(16) Slots {
  uint8_t at[kStages][2][kThreads * 16];
  __device__ __forceinline__ uint8_t *slot(int stage, int i) { return &at[stage][i][threadIdx.x * 16]; }
};

template <typename T>
__device__ __forceinline__ void fetch(Slots *s, int stage, int i, const T *p,
                                      bool on) {
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k)
    pack8::copy_async16(s[k].slot(stage, i), reinterpret_cast<const uint8_t *>(p) + 16 * k, on);
}

template <typename T>
__device__ __forceinline__ void take(Pack8<T> &x, Slots *s, int stage, int i) {
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k)
    x.take(k, *reinterpret_cast<const uint4 *>(s[k].slot(stage, i)));
}

template <typename T, bool GATED>
struct ForwardSmem {
  static constexpr int kV = sizeof(T) / 2;   // 16-byte slots of an element octet
  Slots x[(GATED ? 2 : 1) * kV];         // u, then v
};

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) forward_kernel(const ForwardArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  auto &in = *reinterpret_cast<ForwardSmem<T, GATED> *>(smem);
  const int lane = threadIdx.x & 31;
  const Walk<true> walk(p.T, p.F);
  follow_previous();
  allow_next();
  constexpr int rows = 2;   // from one step to the next
  const int T_rows = (int)p.T, tiles = (int)((p.F + 127) / 128);
  for (int strip = walk.strip; strip < walk.strips; strip += walk.strip_step) {
    const Columns c(strip, p.F);
    int row = 2 * walk.pair0 + (lane >> 4);
    const T *pu = static_cast<const T *>(p.u) + row * p.ldu + c.col;
    const T *pv = static_cast<const T *>(p.v) + (GATED ? row * p.ldv + c.col : 0);
    T *pa = static_cast<T *>(p.a) + row * p.lda + c.col;
    uint8_t *u8 = p.u8 + row * p.F + c.col, *v8 = p.v8 + (GATED ? row * p.F + c.col : 0);
    // scales of the last 16 steps: step k's in lanes k (first row) and 16 + k, so
    // that they leave as 32 neighbouring rows
    float *us = p.u_scales + 2 * (int64_t)strip * p.T, *vs = p.v_scales + (GATED ? 2 * (int64_t)strip * p.T : 0);
    float keep[2][2];
    int next = row;   // row of the next step to fetch
    auto fetch_step = [&](int stage) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = next < T_rows && c.in[i] > 0;
        fetch<T>(in.x, stage, i, on ? pu + 128 * i : static_cast<const T *>(p.u), on);
        if (GATED) fetch<T>(in.x + in.kV, stage, i, on ? pv + 128 * i : static_cast<const T *>(p.v), on);
      }
      pack8::copy_commit();
      next += rows;
      pu += rows * p.ldu;
      if (GATED) pv += rows * p.ldv;
    };
    if (VEC)
      for (int k = 0; k < kStages - 1; ++k) fetch_step(k);
    int stage = 0;
    for (int pair = walk.pair0; pair < walk.pairs; ++pair) {
      Pack8<T> u[2], v[2];
      int valid[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) valid[i] = row < T_rows ? c.in[i] : 0;
      if (VEC) {
        fetch_step(stage == 0 ? kStages - 1 : stage - 1);
        pack8::copy_wait<kStages - 1>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          take<T>(u[i], in.x, stage, i);
          if (GATED) take<T>(v[i], in.x + in.kV, stage, i);
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u[i].load_some(valid[i] > 0 ? pu + 128 * i : static_cast<const T *>(p.u), valid[i]);
          if (GATED) v[i].load_some(valid[i] > 0 ? pv + 128 * i : static_cast<const T *>(p.v), valid[i]);
        }
        pu += rows * p.ldu;
        if (GATED) pv += rows * p.ldv;
      }
      Scales sc;
      find_scales<GATED>(u, v, sc);
      const int k = (pair - walk.pair0) & 15;
      if ((lane & 15) == k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) keep[i][0] = sc.s[i][0], keep[i][1] = sc.s[i][1];
      }
      if (k == 15 || pair == walk.pairs - 1) {
        const int at = 2 * (pair - k + (lane & 15)) + (lane >> 4);
        if ((lane & 15) <= k && at < T_rows) {
          us[at] = keep[0][0];
          if (GATED) vs[at] = keep[0][1];
          if (2 * strip + 1 < tiles) {
            us[p.T + at] = keep[1][0];
            if (GATED) vs[p.T + at] = keep[1][1];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 bu, bv;
        if (sc.finite) {
          bu = cast8(u[i], sc.s[i][0], sc.r[i][0]);
          if (GATED) bv = cast8(v[i], sc.s[i][1], sc.r[i][1]);
        } else {
          bu = cast8_any(u[i], sc.s[i][0], sc.r[i][0]);
          if (GATED) bv = cast8_any(v[i], sc.s[i][1], sc.r[i][1]);
        }
        if (valid[i] > 0) {
          store_bytes<VEC>(u8 + 128 * i, valid[i], bu);
          if (GATED) store_bytes<VEC>(v8 + 128 * i, valid[i], bv);
          float out[8], unused;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            activation<ACT, false>(u[i].at(j), out[j], unused);
            if (GATED) out[j] *= v[i].at(j);
          }
          store<VEC, true>(pa + 128 * i, valid[i], out);
        }
      }
      row += rows;
      pa += rows * p.lda;
      u8 += rows * p.F;
      if (GATED) v8 += rows * p.F;
    }
    if (VEC) pack8::copy_wait<0>();   // the slots are free for the next strip
  }
}

template <int ACT, typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) backward_kernel(const BackwardArgs p) {
  const int lane = threadIdx.x & 31;
  const Walk<false> walk(p.T, p.F);
  follow_previous();
  allow_next();
  const int rows = 2 * walk.step;
  const int T_rows = (int)p.T;
  for (int strip = walk.strip; strip < walk.strips; strip += walk.strip_step) {
    const Columns c(strip, p.F);
    int row = 2 * walk.pair0 + (lane >> 4);
    const T *pd = static_cast<const T *>(p.da) + row * p.ldda + c.col;
    T *pu = static_cast<T *>(p.du) + row * p.lddu + c.col;
    T *pv = static_cast<T *>(p.dv) + (GATED ? row * p.lddv + c.col : 0);
    T *pa = static_cast<T *>(p.a) + row * p.lda + c.col;
    const uint8_t *u8 = p.u8 + row * p.F + c.col, *v8 = p.v8 + (GATED ? row * p.F + c.col : 0);
    const float *us = p.u_scales + 2 * (int64_t)strip * p.T + row;
    const float *vs = p.v_scales + (GATED ? 2 * (int64_t)strip * p.T + row : 0);
    for (int pair = walk.pair0; pair < walk.pairs; pair += walk.step) {
      Pack8<T> d[2];
      uint2 bu[2], bv[2];
      float su[2], sv[2];
      int valid[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        valid[i] = row < T_rows ? c.in[i] : 0;
        if (valid[i] > 0) {
          bu[i] = load_bytes<VEC>(u8 + 128 * i, valid[i]);
          su[i] = us[i * p.T];
          if (GATED) {
            bv[i] = load_bytes<VEC>(v8 + 128 * i, valid[i]);
            sv[i] = vs[i * p.T];
          }
          pack8::load<VEC>(d[i], pd + 128 * i, valid[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (valid[i] == 0) continue;
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
        store<VEC, true>(pu + 128 * i, valid[i], du);
        if (GATED) store<VEC, true>(pv + 128 * i, valid[i], dv);
        if (p.a != nullptr) store<VEC, true>(pa + 128 * i, valid[i], out);
      }
      row += rows;
      pd += rows * p.ldda;
      pu += rows * p.lddu;
      pa += rows * p.lda;
      u8 += rows * p.F;
      us += rows;
      if (GATED) {
        pv += rows * p.lddv;
        v8 += rows * p.F;
        vs += rows;
      }
    }
  }
}

// CTAs that fit on the device at once, no more than there is work for.
template <typename Tag, typename Kernel>
int grid_for(Kernel kernel, int smem, int64_t T, int64_t F) {
  static PerDeviceOnce setup;   // per Tag
  const int fit = setup.get([&] {
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem) != cudaSuccess)
      return 0;
    return n * sm_count();
  });
  const int64_t warps = ((T + 1) / 2) * ((F + 255) / 256);
  return (int)std::min<int64_t>((warps + kThreads / 32 - 1) / (kThreads / 32), fit);
}

bool vec_ok(const void *p, int64_t ld, int64_t size) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0);
}

template <int ACT, typename T, bool GATED, bool VEC>
cudaError_t run_forward(const ForwardArgs &a, cudaStream_t stream) {
  auto kernel = forward_kernel<ACT, T, GATED, VEC>;
  constexpr int smem = VEC ? (int)sizeof(ForwardSmem<T, GATED>) : 0;
  struct Tag {};   // a set-up of its own for every kernel of this signature
  const int grid = grid_for<Tag>(kernel, smem, a.T, a.F);
  if (grid < 1) return cudaErrorInvalidValue;
  log_line("launch act forward_kernel act %d %s%s%s, two rows of 256 columns a warp, grid %d", ACT,
           sizeof(T) == 2 ? "bf16" : "fp32", GATED ? " gated" : "", VEC ? "" : " element by element", grid);
  return Launch((unsigned)grid, 1, kThreads, smem, stream).run(kernel, a);
}

template <int ACT, typename T, bool GATED, bool VEC>
cudaError_t run_backward(const BackwardArgs &a, cudaStream_t stream) {
  auto kernel = backward_kernel<ACT, T, GATED, VEC>;
  constexpr int smem = 0;
  struct Tag {};
  const int grid = grid_for<Tag>(kernel, smem, a.T, a.F);
  if (grid < 1) return cudaErrorInvalidValue;
  log_line("launch act backward_kernel act %d %s%s%s, two rows of 256 columns a warp, grid %d", ACT,
           sizeof(T) == 2 ? "bf16" : "fp32", GATED ? " gated" : "", VEC ? "" : " element by element", grid);
  return Launch((unsigned)grid, 1, kThreads, smem, stream).run(kernel, a);
}

template <int ACT, typename T, bool GATED>
cudaError_t forward(const ForwardArgs &a, bool vec, cudaStream_t stream) {
  return vec ? run_forward<ACT, T, GATED, true>(a, stream) : run_forward<ACT, T, GATED, false>(a, stream);
}

template <int ACT, typename T, bool GATED>
cudaError_t backward(const BackwardArgs &a, bool vec, cudaStream_t stream) {
  return vec ? run_backward<ACT, T, GATED, true>(a, stream)
             : run_backward<ACT, T, GATED, false>(a, stream);
}

template <int ACT>
cudaError_t forward_type(int dtype, const ForwardArgs &a, bool vec, cudaStream_t s) {
  const bool gated = a.v != nullptr;
  if (dtype == FP8Q_DT_BF16)
    return gated ? forward<ACT, __nv_bfloat16, true>(a, vec, s) : forward<ACT, __nv_bfloat16, false>(a, vec, s);
  return gated ? forward<ACT, float, true>(a, vec, s) : forward<ACT, float, false>(a, vec, s);
}

template <int ACT>
cudaError_t backward_type(int dtype, const BackwardArgs &a, bool vec, cudaStream_t s) {
  const bool gated = a.v8 != nullptr;
  if (dtype == FP8Q_DT_BF16)
    return gated ? backward<ACT, __nv_bfloat16, true>(a, vec, s)
          : backward<ACT, __nv_bfloat16, false>(a, vec, s);
  return gated ? backward<ACT, float, true>(a, vec, s) : backward<ACT, float, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_forward(int act, int dtype, const ForwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.F % 16 == 0 && vec_ok(a.u, a.ldu, size) && vec_ok(a.v, a.ldv, size) &&
                   vec_ok(a.a, a.lda, size) && vec_ok(a.u8, a.F, 1) && vec_ok(a.v8, a.F, 1);
  if (act == FP8Q_ACT_SILU)
    return forward_type<FP8Q_ACT_SILU>(dtype, a, vec, stream);
  if (act == FP8Q_ACT_GELU)
    return forward_type<FP8Q_ACT_GELU>(dtype, a, vec, stream);
  return forward_type<FP8Q_ACT_GELU_TANH>(dtype, a, vec, stream);
}

cudaError_t launch_backward(int act, int dtype, const BackwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.F % 16 == 0 && vec_ok(a.u8, a.F, 1) && vec_ok(a.v8, a.F, 1) &&
                   vec_ok(a.da, a.ldda, size) && vec_ok(a.du, a.lddu, size) &&
                   vec_ok(a.dv, a.lddv, size) && vec_ok(a.a, a.lda, size);
  if (act == FP8Q_ACT_SILU)
    return backward_type<FP8Q_ACT_SILU>(dtype, a, vec, stream);
  if (act == FP8Q_ACT_GELU)
    return backward_type<FP8Q_ACT_GELU>(dtype, a, vec, stream);
  return backward_type<FP8Q_ACT_GELU_TANH>(dtype, a, vec, stream);
}

}  // namespace act
}  // namespace fp8q
