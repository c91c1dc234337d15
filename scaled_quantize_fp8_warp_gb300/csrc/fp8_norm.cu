// RMS norm with the residual's addition before it and the E4M3 cast after it,
// and its backward pass:
//   h = round(x + residual), rstd = 1 / sqrt(mean h^2 + eps), y = (h rstd) w,
//   q = RNE_e4m3(y / s), s = max(amax / 448, 1e-12) per 1x128 tile or row;
//   n = h rstd, g = dy w, dx = rstd (g - n mean(g n)) + dresidual,
//   dw = sum over rows of dy n.
// Everything after h's rounding is fp32: h is rounded first because the next
// layer's residual and the backward pass read it as it is stored.
//
// A row is held in registers, eight columns a thread and chunk, by a warp (up to
// 256 columns), by 128 threads (1024), 256 (4096), 512 (forward 16384, backward
// 8192) or 1024, and its successor's loads are under way while it is worked on
// (not by 1024).  A 1x128 tile is a chunk of 16 neighbouring lanes.  Longer rows
// are read again from memory.  Each thread of the backward pass keeps to its
// columns and adds up their part of dw over the rows that its block visits; a
// second launch adds the blocks'.
//
// What bounds it: HBM.  Forward with residual, y and 1x128 tiles, 9.03 bytes an
// element in bf16: 15872 x 4096 93.8 us (6.26 TB/s, 92% of a copy's rate), 65536 x
// 1024 92.6, 4096 x 16384 (row scales) 92.8; fp32 8192 x 4096 104 (5.5).  Backward with
// dresidual, 8 bytes: 8192 x 4096 48.5 us (5.5), of which 2 for adding the blocks'
// sums, 8192 x 8192 88 (6.1), 32768 x 1024 49, 4096 x 16384 126 (4.3: a row's loads wait
// for the row before); fp32 8192 x 4096 98 (5.5), 4096 x 8192 113, 2048 x 16384 111 (4.8).
// Rows that are read again: forward 2048 x 20480 bf16 73 with tile scales and 76 with
// row scales (5.2, 5.0), fp32 1024 x 20480 71; backward 140 both (2.4: dy and h three
// times).  Rows that start anywhere, element by element: 1003 x 2570 fp32 12.6 (1.8),
// 15872 x 4094 bf16 231 (2.6), backward 8192 x 4094 103 (2.6).  The same rows on other numbers of threads, 15872 x 4096
// forward and 8192 x 4096 backward: 512 threads of one chunk 120 and 86, 128 of four
// 112 and 77.  Arithmetic two values at a time (f32x2) took the backward pass from
// 64 to 48.5 us.  One row of 4096: 2.6 us in a graph.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp8_cast8.cuh"
#include "fp8_norm.h"
#include "fp8_pack8.cuh"

namespace fp8q {
namespace norm {
namespace {

using pack8::Pack8;
using tilecast::cast8_any;
using tilecast::store_bytes;
using tilecast::tile_scale;

constexpr unsigned kAll = 0xFFFFFFFFu;

// Threads of a row (RT), and 8-column chunks of each: up to 8 RT CHUNKS columns.
template <int RT, int CHUNKS>
struct Shape {
  static constexpr int kThreads = RT < 256 ? 256 : RT;
  static constexpr int kRows = kThreads / RT;    // rows of a block at once
  static constexpr int kColumns = 8 * RT * CHUNKS;
  // Blocks an SM has to hold: 80 registers a thread forward, 128 backward (80 with one
  // chunk).  Backward in fp32 that is not enough, its rows take twice bf16's registers:
  // 32 to 160 bytes a thread spill, and 96 (bf16) to 180 with 1024 threads.
  static constexpr int kForwardBlocks = CHUNKS > 2 ? 1 : (768 / kThreads > 0 ? 768 / kThreads : 1);
  static constexpr int kBackwardBlocks = kThreads > 512 ? 1 : (CHUNKS == 1 ? 768 : 512) / kThreads;
  // Backward, the next row's loads are under way while one is worked on.  1024
  // threads have no registers for that, nor for the weight's.
  static constexpr bool kAhead = kThreads <= 512;
};

// The eight columns of a thread's chunk (number k of the row's 8-column chunks)
// and how many of them exist.  VEC: neighbours, moved 16 bytes at a time;
// otherwise every 16th of the tile that 16 lanes share, so that lanes move
// neighbouring elements.
template <bool VEC>
struct Columns {
  int64_t first;
  int valid;
  __device__ __forceinline__ Columns(int64_t k, int64_t C) {
    first = VEC ? 8 * k : (k >> 4) * 128 + (k & 15);
    const int64_t left = C - first;
    valid = (int)max((int64_t)0, min((int64_t)8, VEC ? left : (left + 15) >> 4));
    if (valid == 0) first = 0;   // nothing is addressed where nothing is valid
  }
};

// A chunk of a row of T, as pairs of values; zeros past the row.
template <typename T>
struct Raw {
  Pack8<T> x;
  template <bool VEC>
  __device__ __forceinline__ void load(const T *row, const Columns<VEC> &c) {
    const T *p = row + c.first;
    if (VEC) {
      pack8::load<true>(x, p, c.valid);
    } else if constexpr (sizeof(T) == 2) {
      const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x.w[k] = (2 * k < c.valid ? (uint32_t)q[32 * k] : 0u) |
                 (2 * k + 1 < c.valid ? (uint32_t)q[32 * k + 16] << 16 : 0u);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x.v[j] = j < c.valid ? p[16 * j] : 0.0f;
    }
  }
  __device__ __forceinline__ float2 pair(int k) const { return x.pair(k); }
};

template <bool VEC, bool STREAM = false, typename T>
__device__ __forceinline__ void store8(T *row, const Columns<VEC> &c, const float (&v)[8]) {
  if (VEC) {
    pack8::store<true, STREAM>(row + c.first, c.valid, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < c.valid) row[c.first + 16 * j] = (T)v[j];
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_bytes(uint8_t *row, const Columns<VEC> &c, uint2 w) {
  if (VEC) {
    store_bytes<true>(row + c.first, c.valid, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < c.valid) row[c.first + 16 * j] = (uint8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * (j - 4))) & 0xFFu);
  }
}

// A chunk of the weight.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void *w, int w_bf16, const Columns<VEC> &c, float2 (&out)[4]) {
  if (w_bf16) {
    Raw<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16 *>(w), c);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = r.pair(k);
  } else {
    Raw<float> r;
    r.load(static_cast<const float *>(w), c);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = r.pair(k);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Sum and maximum over a row's threads, the same in each; a row's warps meet in
// a slot of shared memory that the next but one call uses again, at a barrier of
// their own.
template <int RT>
struct Reduce {
  float (*slot)[RT / 32];
  int turn = 0;
  __device__ __forceinline__ void meet() const {
    if (RT >= 256)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / RT), "n"(RT) : "memory");
  }
  __device__ __forceinline__ float sum(float v) {
    v = warp_sum(v);
    if constexpr (RT == 32) return v;
    float *s = slot[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x % RT) >> 5] = v;
    meet();
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < RT / 32; ++k) v += s[k];
    return v;
  }
  __device__ __forceinline__ uint32_t max_bits(uint32_t v) {
    v = __reduce_max_sync(kAll, v);
    if constexpr (RT == 32) return v;
    float *s = slot[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x % RT) >> 5] = __uint_as_float(v);
    meet();
    v = 0u;
#pragma unroll
    for (int k = 0; k < RT / 32; ++k) v = max(v, __float_as_uint(s[k]));
    return v;
  }
};

// The rounded sum x + r, as the values that are stored.
template <typename T>
__device__ __forceinline__ void add_rounded(const Raw<T> &x, const Raw<T> &r, float2 (&h)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = __fadd2_rn(x.pair(k), r.pair(k));
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = pack8::bf16x2(h[k].x, h[k].y);
      h[k] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
  }
}
__device__ __forceinline__ void spread(const float2 (&v)[4], float (&out)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) out[2 * k] = v[k].x, out[2 * k + 1] = v[k].y;
}
// y = (v rstd) w.
__device__ __forceinline__ void normed(const float2 (&v)[4], float rstd, const float2 (&w)[4], Pack8<float> &y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = __fmul2_rn(__fmul2_rn(v[k], make_float2(rstd, rstd)), w[k]);
    y.v[2 * k] = t.x, y.v[2 * k + 1] = t.y;
  }
}

__device__ __forceinline__ float rstd_of(float sum, const ForwardArgs &p) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.C), p.eps));
}

// max |y| of the 16 lanes that hold a tile.
__device__ __forceinline__ uint32_t tile_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
  return m;
}

template <typename T, int RT, int CHUNKS, bool VEC>
__global__ void __launch_bounds__(Shape<RT, CHUNKS>::kThreads, Shape<RT, CHUNKS>::kForwardBlocks)
    forward_kernel(const ForwardArgs p) {
  using S = Shape<RT, CHUNKS>;
  __shared__ float slots[S::kRows][2][RT / 32];
  Reduce<RT> reduce{slots[threadIdx.x / RT]};
  const int t = threadIdx.x % RT;
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  int64_t row = (int64_t)blockIdx.x * S::kRows + threadIdx.x / RT;
  follow_previous();
  allow_next();
  float2 w[CHUNKS][4];
  const auto at = [&](int i) { return Columns<VEC>(i * RT + t, p.C); };
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) load_weight(p.weight, p.w_bf16, at(i), w[i]);
  const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
  Raw<T> a[CHUNKS], b[CHUNKS];
  const auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      a[i].load(x + r * p.ldx, at(i));
      if (res != nullptr) b[i].load(res + r * p.ldr, at(i));
    }
  };
  if (row < p.T) fetch(row);
  for (; row < p.T; row += step) {
    float2 v[CHUNKS][4], sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      if (res != nullptr) {
        add_rounded<T>(a[i], b[i], v[i]);
        float h[8];
        spread(v[i], h);
        store8(static_cast<T *>(p.h) + row * p.ldh, at(i), h);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = a[i].pair(k);
      }
    }
    if (row + step < p.T) fetch(row + step);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = __ffma2_rn(v[i][k], v[i][k], sum);
    const float rstd = rstd_of(reduce.sum(sum.x + sum.y), p);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    uint32_t m[CHUNKS], all = 0u;
    Pack8<float> y[CHUNKS];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      normed(v[i], rstd, w[i], y[i]);
      if (p.y != nullptr) store8<VEC, true>(static_cast<T *>(p.y) + row * p.ldy, at(i), y[i].v);
      m[i] = y[i].amax_bits();
      all = max(all, m[i]);
    }
    if (p.q == nullptr) continue;
    float s = 0.0f;
    if (p.row_scale) {
      s = tile_scale(reduce.max_bits(all));
      if (t == 0) p.q_scales[row] = s;
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      if (!p.row_scale) {
        s = tile_scale(tile_max(m[i]));
        const int64_t tile = (i * RT + t) >> 4;
        if ((t & 15) == 0 && 128 * tile < p.C) p.q_scales[tile * p.T + row] = s;
      }
      store8_bytes(p.q + row * p.C, at(i), cast8_any(y[i], s, __frcp_rn(s)));
    }
  }
}

// Rows longer than the registers hold: read again for every pass.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) forward_long_kernel(const ForwardArgs p) {
  constexpr int RT = 512;
  __shared__ float slots[2][RT / 32];
  Reduce<RT> reduce{slots};
  const int t = threadIdx.x;
  follow_previous();
  allow_next();
  const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
  const int64_t chunks = (p.C + 127) / 128 * 16;   // whole tiles
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    float2 sum = make_float2(0.0f, 0.0f);
    for (int64_t k = t; k < chunks; k += RT) {
      const Columns<VEC> at(k, p.C);
      Raw<T> a, b;
      float2 v[4];
      a.load(x + row * p.ldx, at);
      if (res != nullptr) {
        b.load(res + row * p.ldr, at);
        add_rounded<T>(a, b, v);
        float h[8];
        spread(v, h);
        store8(static_cast<T *>(p.h) + row * p.ldh, at, h);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a.pair(j);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = __ffma2_rn(v[j], v[j], sum);
    }
    const float rstd = rstd_of(reduce.sum(sum.x + sum.y), p);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    // what this thread stored as h, or x where there is no residual
    const T *h = res != nullptr ? static_cast<const T *>(p.h) + row * p.ldh : x + row * p.ldx;
    const auto read = [&](const Columns<VEC> &at, Pack8<float> &y) {
      Raw<T> a;
      float2 v[4], w[4];
      a.load(h, at);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a.pair(j);
      load_weight(p.weight, p.w_bf16, at, w);
      normed(v, rstd, w, y);
    };
    uint32_t all = 0u;
    const bool cast = p.q != nullptr && !p.row_scale;
    for (int64_t k0 = 0; k0 < chunks; k0 += RT) {   // whole warps, for the tiles' maxima
      const Columns<VEC> at(k0 + t, p.C);
      Pack8<float> y;
      read(at, y);
      if (p.y != nullptr) store8<VEC, true>(static_cast<T *>(p.y) + row * p.ldy, at, y.v);
      const uint32_t m = y.amax_bits();
      all = max(all, m);
      if (!cast) continue;
      const float s = tile_scale(tile_max(m));
      if ((t & 15) == 0 && 8 * (k0 + t) < p.C) p.q_scales[((k0 + t) >> 4) * p.T + row] = s;
      store8_bytes(p.q + row * p.C, at, cast8_any(y, s, __frcp_rn(s)));
    }
    if (p.q == nullptr || cast) continue;
    const float s = tile_scale(reduce.max_bits(all)), r = __frcp_rn(s);
    if (t == 0) p.q_scales[row] = s;
    for (int64_t k = t; k < chunks; k += RT) {
      const Columns<VEC> at(k, p.C);
      Pack8<float> y;
      read(at, y);
      store8_bytes(p.q + row * p.C, at, cast8_any(y, s, r));
    }
  }
}

// n = h rstd and g = dy w of one chunk.
template <typename T>
__device__ __forceinline__ void terms(const Raw<T> &dy, const Raw<T> &h, float rstd, const float2 (&w)[4],
                                      float2 (&g)[4], float2 (&n)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    n[k] = __fmul2_rn(h.pair(k), make_float2(rstd, rstd));
    g[k] = __fmul2_rn(dy.pair(k), w[k]);
  }
}

// dx = rstd (g - n mean) + dresidual of one chunk.
template <bool VEC, typename T>
__device__ __forceinline__ void store_dx(const BackwardArgs &p, int64_t row, const Columns<VEC> &at,
                                         const float2 (&g)[4], const float2 (&n)[4], float mean, float rstd,
                                         const Raw<T> &add) {
  float2 dx[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    dx[k] = __fmul2_rn(make_float2(rstd, rstd), __ffma2_rn(n[k], make_float2(-mean, -mean), g[k]));
    if (p.dresidual != nullptr) dx[k] = __fadd2_rn(dx[k], add.pair(k));
  }
  float out[8];
  spread(dx, out);
  store8<VEC, true>(static_cast<T *>(p.dx) + row * p.lddx, at, out);
}

template <typename T, int RT, int CHUNKS, bool VEC>
__global__ void __launch_bounds__(Shape<RT, CHUNKS>::kThreads, Shape<RT, CHUNKS>::kBackwardBlocks)
    backward_kernel(const BackwardArgs p) {
  using S = Shape<RT, CHUNKS>;
  __shared__ float slots[S::kRows][2][RT / 32];
  __shared__ __align__(16) float join[S::kRows > 1 ? S::kRows : 1][S::kRows > 1 ? S::kColumns : 1];
  Reduce<RT> reduce{slots[threadIdx.x / RT]};
  const int t = threadIdx.x % RT, mine = threadIdx.x / RT;
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  int64_t row = (int64_t)blockIdx.x * S::kRows + mine;
  follow_previous();
  allow_next();
  const T *dy = static_cast<const T *>(p.dy), *h = static_cast<const T *>(p.h);
  const T *res = static_cast<const T *>(p.dresidual);
  const auto at = [&](int i) { return Columns<VEC>(i * RT + t, p.C); };
  float2 dw[CHUNKS][4], w[CHUNKS][4];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    if (S::kAhead) load_weight(p.weight, p.w_bf16, at(i), w[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = make_float2(0.0f, 0.0f);
  }
  Raw<T> a[CHUNKS], b[CHUNKS], add[CHUNKS];   // dy, h, dresidual of the next row
  float rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      a[i].load(dy + r * p.lddy, at(i));
      b[i].load(h + r * p.ldh, at(i));
      if (S::kAhead && res != nullptr) add[i].load(res + r * p.lddr, at(i));
    }
    rstd = p.rstd[r];
  };
  if (S::kAhead && row < p.T) fetch(row);
  for (; row < p.T; row += step) {
    // this row stays as it was read, half the registers of bf16's values: n and
    // g are found twice
    if (!S::kAhead) fetch(row);
    Raw<T> d[CHUNKS], x[CHUNKS], plus[CHUNKS];
    const float scale = rstd;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) d[i] = a[i], x[i] = b[i], plus[i] = add[i];
    if (S::kAhead && row + step < p.T) fetch(row + step);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      float2 g[4], n[4];
      if (!S::kAhead) load_weight(p.weight, p.w_bf16, at(i), w[i]);
      terms(d[i], x[i], scale, w[i], g, n);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dw[i][k] = __ffma2_rn(d[i].pair(k), n[k], dw[i][k]);
        sum = __ffma2_rn(g[k], n[k], sum);
      }
    }
    const float mean = __fdiv_rn(reduce.sum(sum.x + sum.y), (float)p.C);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      float2 g[4], n[4];
      if (!S::kAhead) {
        load_weight(p.weight, p.w_bf16, at(i), w[i]);
        if (res != nullptr) plus[i].load(res + row * p.lddr, at(i));
      }
      terms(d[i], x[i], scale, w[i], g, n);
      store_dx(p, row, at(i), g, n, mean, scale, plus[i]);
    }
  }
  if (p.dweight == nullptr) return;
  float *out = p.partial + (int64_t)blockIdx.x * p.C;
  if constexpr (S::kRows > 1) {   // the warps' sums, added in their order
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      float v[8];
      spread(dw[i], v);
      store8(join[mine], at(i), v);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (int)p.C; c += S::kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < S::kRows; ++k) s += join[k][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      float v[8];
      spread(dw[i], v);
      store8(out, at(i), v);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(512) backward_long_kernel(const BackwardArgs p) {
  constexpr int RT = 512;
  __shared__ float slots[2][RT / 32];
  Reduce<RT> reduce{slots};
  const int64_t t = threadIdx.x, chunks = (p.C + 127) / 128 * 16;
  follow_previous();
  allow_next();
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const float rstd = p.rstd[row];
    float2 g[4], n[4], sum = make_float2(0.0f, 0.0f);
    const auto read = [&](const Columns<VEC> &at) {
      Raw<T> a, b;
      float2 w[4];
      a.load(static_cast<const T *>(p.dy) + row * p.lddy, at);
      b.load(static_cast<const T *>(p.h) + row * p.ldh, at);
      load_weight(p.weight, p.w_bf16, at, w);
      terms(a, b, rstd, w, g, n);
    };
    for (int64_t k = t; k < chunks; k += RT) {
      read(Columns<VEC>(k, p.C));
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = __ffma2_rn(g[j], n[j], sum);
    }
    const float mean = __fdiv_rn(reduce.sum(sum.x + sum.y), (float)p.C);
    for (int64_t k = t; k < chunks; k += RT) {
      const Columns<VEC> at(k, p.C);
      read(at);
      Raw<T> add;
      if (p.dresidual != nullptr) add.load(static_cast<const T *>(p.dresidual) + row * p.lddr, at);
      store_dx(p, row, at, g, n, mean, rstd, add);
    }
  }
}

// dw's partial sums where rows are too long for backward_kernel: a column a
// thread, rows y, y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) columns_kernel(const BackwardArgs p) {
  follow_previous();
  allow_next();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.C) return;
  float sum = 0.0f;
  for (int64_t row = blockIdx.y; row < p.T; row += gridDim.y) {
    const float n = __fmul_rn((float)static_cast<const T *>(p.h)[row * p.ldh + c], p.rstd[row]);
    sum = fmaf((float)static_cast<const T *>(p.dy)[row * p.lddy + c], n, sum);
  }
  p.partial[(int64_t)blockIdx.y * p.C + c] = sum;
}

// dweight from `count` rows of partial sums: 32 columns a block, whose warps
// take the rows in turns and are added in their order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const float *partial, int count, int64_t C,
                                                               void *dweight, int w_bf16) {
  __shared__ float sums[kJoinWarps][33];
  follow_previous();
  allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 10
    for (int k = warp; k < count; k += kJoinWarps) s += partial[k * C + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= C) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) s += sums[k][lane];
  if (w_bf16)
    static_cast<__nv_bfloat16 *>(dweight)[c] = __float2bfloat16_rn(s);
  else
    static_cast<float *>(dweight)[c] = s;
}

// Blocks of a kernel that fit on the device at once.
template <typename Tag, typename Kernel>
int fitting(Kernel kernel, int threads) {
  static PerDeviceOnce setup;   // per Tag
  return setup.get([&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) return 0;
    return n * sm_count();
  });
}

template <typename T, int RT, int CHUNKS, bool VEC>
cudaError_t run_forward(const ForwardArgs &a, cudaStream_t stream) {
  using S = Shape<RT, CHUNKS>;
  auto kernel = forward_kernel<T, RT, CHUNKS, VEC>;
  struct Tag {};
  const int fit = fitting<Tag>(kernel, S::kThreads);
  if (fit < 1) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>((a.T + S::kRows - 1) / S::kRows, fit);
  log_line("launch norm forward_kernel %s%s, %d threads x %d chunks a row, grid %d",
           sizeof(T) == 2 ? "bf16" : "fp32", VEC ? "" : " element by element", RT, CHUNKS, grid);
  return Launch((unsigned)grid, 1, S::kThreads, 0, stream).run(kernel, a);
}

template <typename T, bool VEC>
cudaError_t forward(const ForwardArgs &a, cudaStream_t stream) {
  if (a.C <= 256) return run_forward<T, 32, 1, VEC>(a, stream);
  if (a.C <= 1024) return run_forward<T, 128, 1, VEC>(a, stream);
  if (a.C <= 2048) return run_forward<T, 256, 1, VEC>(a, stream);
  if (a.C <= 4096) return run_forward<T, 256, 2, VEC>(a, stream);
  if (a.C <= 8192) return run_forward<T, 512, 2, VEC>(a, stream);
  if (a.C <= 16384) return run_forward<T, 512, 4, VEC>(a, stream);
  auto kernel = forward_long_kernel<T, VEC>;
  struct Tag {};
  const int fit = fitting<Tag>(kernel, 512);
  if (fit < 1) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>(a.T, fit);
  log_line("launch norm forward_long_kernel %s%s, grid %d", sizeof(T) == 2 ? "bf16" : "fp32",
           VEC ? "" : " element by element", grid);
  return Launch((unsigned)grid, 1, 512, 0, stream).run(kernel, a);
}

template <typename T, int RT, int CHUNKS, bool VEC>
cudaError_t run_backward(const BackwardArgs &a, int &partials, cudaStream_t stream) {
  using S = Shape<RT, CHUNKS>;
  auto kernel = backward_kernel<T, RT, CHUNKS, VEC>;
  struct Tag {};
  const int fit = std::min(fitting<Tag>(kernel, S::kThreads), kPartials);
  if (fit < 1) return cudaErrorInvalidValue;
  partials = (int)std::min<int64_t>((a.T + S::kRows - 1) / S::kRows, fit);
  log_line("launch norm backward_kernel %s%s, %d threads x %d chunks a row, grid %d",
           sizeof(T) == 2 ? "bf16" : "fp32", VEC ? "" : " element by element", RT, CHUNKS, partials);
  return Launch((unsigned)partials, 1, S::kThreads, 0, stream).run(kernel, a);
}

template <typename T, bool VEC>
cudaError_t backward(const BackwardArgs &a, int &partials, cudaStream_t stream) {
  if (a.C <= 256) return run_backward<T, 32, 1, VEC>(a, partials, stream);
  if (a.C <= 1024) return run_backward<T, 128, 1, VEC>(a, partials, stream);
  if (a.C <= 2048) return run_backward<T, 256, 1, VEC>(a, partials, stream);
  if (a.C <= 4096) return run_backward<T, 256, 2, VEC>(a, partials, stream);
  if (a.C <= 8192) return run_backward<T, 512, 2, VEC>(a, partials, stream);
  if (a.C <= 16384) return run_backward<T, 1024, 2, VEC>(a, partials, stream);
  // dw first: dx may overwrite dy
  if (a.dweight != nullptr) {
    const int64_t columns = (a.C + 255) / 256;
    partials = (int)std::min<int64_t>(std::min<int64_t>(a.T, kPartials), 65535);
    log_line("launch norm columns_kernel, grid %lld x %d", (long long)columns, partials);
    const cudaError_t e =
        Launch((unsigned)columns, (unsigned)partials, 256, 0, stream).run(columns_kernel<T>, a);
    if (e != cudaSuccess) return e;
  }
  auto kernel = backward_long_kernel<T, VEC>;
  struct Tag {};
  const int fit = fitting<Tag>(kernel, 512);
  if (fit < 1) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>(a.T, fit);
  log_line("launch norm backward_long_kernel %s%s, grid %d", sizeof(T) == 2 ? "bf16" : "fp32",
           VEC ? "" : " element by element", grid);
  return Launch((unsigned)grid, 1, 512, 0, stream).run(kernel, a);
}

bool rows_aligned(const void *p, int64_t ld, int64_t size) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0);
}

}  // namespace

cudaError_t launch_forward(int dtype, const ForwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.C % 8 == 0 && rows_aligned(a.x, a.ldx, size) &&
                   rows_aligned(a.residual, a.ldr, size) && rows_aligned(a.h, a.ldh, size) &&
                   rows_aligned(a.y, a.ldy, size) && rows_aligned(a.weight, 0, 1) &&
                   (reinterpret_cast<uintptr_t>(a.q) & 7u) == 0;
  if (dtype == FP8Q_DT_BF16)
    return vec ? forward<__nv_bfloat16, true>(a, stream) : forward<__nv_bfloat16, false>(a, stream);
  return vec ? forward<float, true>(a, stream) : forward<float, false>(a, stream);
}

cudaError_t launch_backward(int dtype, const BackwardArgs &a, cudaStream_t stream) {
  const int64_t size = dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = a.C % 8 == 0 && rows_aligned(a.dy, a.lddy, size) && rows_aligned(a.h, a.ldh, size) &&
                   rows_aligned(a.dresidual, a.lddr, size) && rows_aligned(a.dx, a.lddx, size) &&
                   rows_aligned(a.weight, 0, 1);
  int partials = 0;
  if (a.T > 0) {
    cudaError_t e;
    if (dtype == FP8Q_DT_BF16)
      e = vec ? backward<__nv_bfloat16, true>(a, partials, stream)
              : backward<__nv_bfloat16, false>(a, partials, stream);
    else
      e = vec ? backward<float, true>(a, partials, stream) : backward<float, false>(a, partials, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr) return cudaSuccess;
  const int64_t blocks = (a.C + 31) / 32;
  log_line("launch norm join_kernel, %d partial sums, grid %lld", partials, (long long)blocks);
  return Launch((unsigned)blocks, 1, 32 * kJoinWarps, 0, stream)
      .run(join_kernel, static_cast<const float *>(a.partial), partials, a.C, a.dweight, a.w_bf16);
}

}  // namespace norm
}  // namespace fp8q
