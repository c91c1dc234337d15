// RMS norm with the residual's addition before it and the E4M3 cast after it,
// and its backward pass:
//   h = round(x + residual), rstd = 1 / sqrt(mean h^2 + eps), y = (h rstd) w,
//   q = RNE_e4m3(y / s), s = max(amax / 448, 1e-12) per 1x128 tile or row;
//   n = h rstd, g = dy w, dx = rstd (g - n mean(g n)) + dresidual,
//   dw = sum over rows of dy n.
// Everything after h's rounding is fp32: h is rounded first because the next
// layer's residual and the backward pass read it as it is stored.
//
// A row is held in registers by a warp (up to 1024 columns) or by a block of
// 256 or 512 threads (up to 16384), eight columns a thread and chunk, and its
// successor's loads are under way while it is worked on.  A 1x128 tile is a
// chunk of 16 neighbouring lanes.  Longer rows are read again from memory.
// Each thread of the backward pass keeps to its columns and adds up their part
// of dw over the rows that its block visits; a second launch adds the blocks'.
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
using pack8::store;
using tilecast::cast8_any;
using tilecast::store_bytes;
using tilecast::tile_scale;

constexpr unsigned kAll = 0xFFFFFFFFu;

// Threads of a row, and 8-column chunks of each: rows of up to 8 RT CHUNKS.
template <int RT, int CHUNKS>
struct Shape {
  static constexpr int kThreads = RT < 256 ? 256 : RT;
  static constexpr int kRows = kThreads / RT;    // rows of a block at once
  static constexpr int kColumns = 8 * RT * CHUNKS;
};

__device__ __forceinline__ int columns_in(int64_t col, int64_t C) {
  return (int)max((int64_t)0, min((int64_t)8, C - col));
}

// Eight weights from column c on; zeros past the row.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void *w, int w_bf16, int64_t c, int valid,
                                            float (&out)[8]) {
  if (w_bf16) {
    Pack8<__nv_bfloat16> p;
    pack8::load<VEC>(p, static_cast<const __nv_bfloat16 *>(w) + (valid > 0 ? c : 0), valid);
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = p.at(j);
  } else {
    Pack8<float> p;
    pack8::load<VEC>(p, static_cast<const float *>(w) + (valid > 0 ? c : 0), valid);
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = p.at(j);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Sum and maximum over a row's threads, the same in each; the block's warps
// meet in a slot of shared memory that the next but one call uses again.
template <int RT>
struct Reduce {
  float (*slot)[RT / 32];
  int turn = 0;
  __device__ __forceinline__ float sum(float v) {
    v = warp_sum(v);
    if constexpr (RT == 32) return v;
    float *s = slot[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
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
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = __uint_as_float(v);
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int k = 0; k < RT / 32; ++k) v = max(v, __float_as_uint(s[k]));
    return v;
  }
};

// The rounded sum x + r, as the values that are stored.
template <typename T>
__device__ __forceinline__ void add_rounded(const Pack8<T> &x, const Pack8<T> &r, float (&h)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = __fadd_rn(x.at(j), r.at(j));
    if constexpr (sizeof(T) == 2) h[j] = __bfloat162float(__float2bfloat16_rn(h[j]));
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
__global__ void __launch_bounds__(Shape<RT, CHUNKS>::kThreads) forward_kernel(const ForwardArgs p) {
  using S = Shape<RT, CHUNKS>;
  __shared__ float slots[2][RT / 32];
  Reduce<RT> reduce{slots};
  const int t = threadIdx.x % RT;
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  int64_t row = (int64_t)blockIdx.x * S::kRows + threadIdx.x / RT;
  follow_previous();
  allow_next();
  float w[CHUNKS][8];
  int valid[CHUNKS];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int64_t c = 8 * (int64_t)(i * RT + t);
    valid[i] = columns_in(c, p.C);
    load_weight<VEC>(p.weight, p.w_bf16, c, valid[i], w[i]);
  }
  const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
  Pack8<T> a[CHUNKS], b[CHUNKS];
  const auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int64_t c = valid[i] > 0 ? 8 * (int64_t)(i * RT + t) : 0;
      pack8::load<VEC>(a[i], x + r * p.ldx + c, valid[i]);
      if (res != nullptr) pack8::load<VEC>(b[i], res + r * p.ldr + c, valid[i]);
    }
  };
  if (row < p.T) fetch(row);
  for (; row < p.T; row += step) {
    float v[CHUNKS][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int64_t c = 8 * (int64_t)(i * RT + t);
      if (res != nullptr) {
        add_rounded<T>(a[i], b[i], v[i]);
        store<VEC>(static_cast<T *>(p.h) + row * p.ldh + c, valid[i], v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = a[i].at(j);
      }
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    if (row + step < p.T) fetch(row + step);
    const float rstd = rstd_of(reduce.sum(sum), p);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    uint32_t m[CHUNKS], all = 0u;
    Pack8<float> y[CHUNKS];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i].v[j] = __fmul_rn(__fmul_rn(v[i][j], rstd), w[i][j]);
      if (p.y != nullptr)
        store<VEC>(static_cast<T *>(p.y) + row * p.ldy + 8 * (int64_t)(i * RT + t), valid[i], y[i].v);
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
      const int64_t c = 8 * (int64_t)(i * RT + t);
      if (!p.row_scale) {
        s = tile_scale(tile_max(m[i]));
        if ((t & 15) == 0 && valid[i] > 0) p.q_scales[(c >> 7) * p.T + row] = s;
      }
      store_bytes<VEC>(p.q + row * p.C + c, valid[i], cast8_any(y[i], s, __frcp_rn(s)));
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
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    float sum = 0.0f;
    for (int64_t c = 8 * t; c < p.C; c += 8 * RT) {
      const int valid = columns_in(c, p.C);
      Pack8<T> a, b;
      float v[8];
      pack8::load<VEC>(a, x + row * p.ldx + c, valid);
      if (res != nullptr) {
        pack8::load<VEC>(b, res + row * p.ldr + c, valid);
        add_rounded<T>(a, b, v);
        store<VEC>(static_cast<T *>(p.h) + row * p.ldh + c, valid, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a.at(j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
    }
    const float rstd = rstd_of(reduce.sum(sum), p);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    // what this thread stored as h, or x where there is no residual
    const T *h = res != nullptr ? static_cast<const T *>(p.h) + row * p.ldh : x + row * p.ldx;
    const auto normed = [&](int64_t c, int valid, Pack8<float> &y) {
      Pack8<T> a;
      float w[8];
      pack8::load<VEC>(a, h + (valid > 0 ? c : 0), valid);
      load_weight<VEC>(p.weight, p.w_bf16, c, valid, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y.v[j] = __fmul_rn(__fmul_rn(a.at(j), rstd), w[j]);
    };
    uint32_t all = 0u;
    const bool cast = p.q != nullptr && !p.row_scale;
    for (int64_t c0 = 0; c0 < p.C; c0 += 8 * RT) {   // whole warps, for the tiles' maxima
      const int64_t c = c0 + 8 * t;
      const int valid = columns_in(c, p.C);
      Pack8<float> y;
      normed(c, valid, y);
      if (p.y != nullptr) store<VEC>(static_cast<T *>(p.y) + row * p.ldy + c, valid, y.v);
      const uint32_t m = y.amax_bits();
      all = max(all, m);
      if (!cast) continue;
      const float s = tile_scale(tile_max(m));
      if ((t & 15) == 0 && valid > 0) p.q_scales[(c >> 7) * p.T + row] = s;
      store_bytes<VEC>(p.q + row * p.C + c, valid, cast8_any(y, s, __frcp_rn(s)));
    }
    if (p.q == nullptr || cast) continue;
    const float s = tile_scale(reduce.max_bits(all)), r = __frcp_rn(s);
    if (t == 0) p.q_scales[row] = s;
    for (int64_t c = 8 * t; c < p.C; c += 8 * RT) {
      const int valid = columns_in(c, p.C);
      Pack8<float> y;
      normed(c, valid, y);
      store_bytes<VEC>(p.q + row * p.C + c, valid, cast8_any(y, s, r));
    }
  }
}

// dx of one chunk.
template <typename T, bool VEC>
__device__ __forceinline__ void store_dx(const BackwardArgs &p, int64_t row, int64_t c, int valid,
                                         const float (&g)[8], const float (&n)[8], float mean,
                                         float rstd, const Pack8<T> &add) {
  float dx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dx[j] = __fmul_rn(rstd, fmaf(-n[j], mean, g[j]));
    if (p.dresidual != nullptr) dx[j] = __fadd_rn(dx[j], add.at(j));
  }
  store<VEC>(static_cast<T *>(p.dx) + row * p.lddx + c, valid, dx);
}

template <typename T, int RT, int CHUNKS, bool VEC>
__global__ void __launch_bounds__(Shape<RT, CHUNKS>::kThreads) backward_kernel(const BackwardArgs p) {
  using S = Shape<RT, CHUNKS>;
  __shared__ float slots[2][RT / 32];
  __shared__ float join[S::kRows > 1 ? S::kRows : 1][S::kRows > 1 ? S::kColumns : 1];
  Reduce<RT> reduce{slots};
  const int t = threadIdx.x % RT, mine = threadIdx.x / RT;
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  int64_t row = (int64_t)blockIdx.x * S::kRows + mine;
  follow_previous();
  allow_next();
  const T *dy = static_cast<const T *>(p.dy), *h = static_cast<const T *>(p.h);
  const T *res = static_cast<const T *>(p.dresidual);
  int valid[CHUNKS];
  float dw[CHUNKS][8];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    valid[i] = columns_in(8 * (int64_t)(i * RT + t), p.C);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  Pack8<T> a[CHUNKS], b[CHUNKS];
  float rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int64_t c = valid[i] > 0 ? 8 * (int64_t)(i * RT + t) : 0;
      pack8::load<VEC>(a[i], dy + r * p.lddy + c, valid[i]);
      pack8::load<VEC>(b[i], h + r * p.ldh + c, valid[i]);
    }
    rstd = p.rstd[r];
  };
  if (row < p.T) fetch(row);
  for (; row < p.T; row += step) {
    float g[CHUNKS][8], n[CHUNKS][8];
    Pack8<T> add[CHUNKS];
    const float scale = rstd;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int64_t c = 8 * (int64_t)(i * RT + t);
      float w[8];
      load_weight<VEC>(p.weight, p.w_bf16, c, valid[i], w);
      if (res != nullptr) pack8::load<VEC>(add[i], res + row * p.lddr + (valid[i] > 0 ? c : 0), valid[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = a[i].at(j);
        n[i][j] = __fmul_rn(b[i].at(j), scale);
        g[i][j] = __fmul_rn(d, w[j]);
        dw[i][j] = fmaf(d, n[i][j], dw[i][j]);
        sum = fmaf(g[i][j], n[i][j], sum);
      }
    }
    if (row + step < p.T) fetch(row + step);
    const float mean = __fdiv_rn(reduce.sum(sum), (float)p.C);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
      store_dx<T, VEC>(p, row, 8 * (int64_t)(i * RT + t), valid[i], g[i], n[i], mean, scale, add[i]);
  }
  if (p.dweight == nullptr) return;
  float *out = p.partial + (int64_t)blockIdx.x * p.C;
  if constexpr (S::kRows > 1) {   // the warps' sums, added in their order
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) join[mine][8 * (i * RT + t) + j] = dw[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < (int)p.C; c += S::kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < S::kRows; ++k) s += join[k][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid[i]) out[8 * (int64_t)(i * RT + t) + j] = dw[i][j];
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(512) backward_long_kernel(const BackwardArgs p) {
  constexpr int RT = 512;
  __shared__ float slots[2][RT / 32];
  Reduce<RT> reduce{slots};
  const int t = threadIdx.x;
  follow_previous();
  allow_next();
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const float rstd = p.rstd[row];
    float g[8], n[8];
    const auto read = [&](int64_t c, int valid) {
      Pack8<T> a, b;
      float w[8];
      pack8::load<VEC>(a, static_cast<const T *>(p.dy) + row * p.lddy + c, valid);
      pack8::load<VEC>(b, static_cast<const T *>(p.h) + row * p.ldh + c, valid);
      load_weight<VEC>(p.weight, p.w_bf16, c, valid, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] = __fmul_rn(b.at(j), rstd);
        g[j] = __fmul_rn(a.at(j), w[j]);
      }
    };
    float sum = 0.0f;
    for (int64_t c = 8 * t; c < p.C; c += 8 * RT) {
      read(c, columns_in(c, p.C));
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(g[j], n[j], sum);
    }
    const float mean = __fdiv_rn(reduce.sum(sum), (float)p.C);
    for (int64_t c = 8 * t; c < p.C; c += 8 * RT) {
      const int valid = columns_in(c, p.C);
      read(c, valid);
      Pack8<T> add;
      if (p.dresidual != nullptr)
        pack8::load<VEC>(add, static_cast<const T *>(p.dresidual) + row * p.lddr + c, valid);
      store_dx<T, VEC>(p, row, c, valid, g, n, mean, rstd, add);
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

// dweight from `count` rows of partial sums: 32 columns a block, whose eight
// warps take the rows in turns and are added in their order.
__global__ void __launch_bounds__(256) join_kernel(const float *partial, int count, int64_t C,
                                                   void *dweight, int w_bf16) {
  __shared__ float sums[8][33];
  follow_previous();
  allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int k = warp; k < count; k += 8) s += partial[k * C + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= C) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += sums[k][lane];
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
  if (a.C <= 1024) return run_forward<T, 32, 4, VEC>(a, stream);
  if (a.C <= 2048) return run_forward<T, 256, 1, VEC>(a, stream);
  if (a.C <= 4096) return run_forward<T, 256, 2, VEC>(a, stream);
  if (a.C <= 8192) return run_forward<T, 256, 4, VEC>(a, stream);
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
  if (a.C <= 1024) return run_backward<T, 32, 4, VEC>(a, partials, stream);
  if (a.C <= 2048) return run_backward<T, 256, 1, VEC>(a, partials, stream);
  if (a.C <= 4096) return run_backward<T, 256, 2, VEC>(a, partials, stream);
  if (a.C <= 8192) return run_backward<T, 512, 2, VEC>(a, partials, stream);
  if (a.C <= 16384) return run_backward<T, 512, 4, VEC>(a, partials, stream);
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
  return Launch((unsigned)blocks, 1, 256, 0, stream)
      .run(join_kernel, static_cast<const float *>(a.partial), partials, a.C, a.dweight, a.w_bf16);
}

}  // namespace norm
}  // namespace fp8q
