// 4-bit quantisation (MXFP4, NVFP4) and its inverse.
//
// quantize_kernel: a CTA of 256 threads owns a 128 x 128 tile of x.  Warp w
// holds rows [32 (w / 2), +32) and columns [64 (w % 2), +64); lane l the rows
// [8 (l / 8), +8) and columns [8 (l % 8), +8) of that, so a block of 32 (or
// 16) along a row lies in 4 (2) neighbouring lanes and a block of 32 (16) down
// a column in 4 (2) lanes eight apart: both maxima are butterflies inside the
// warp.  One read of x serves both orientations; each is cast with its own
// scales.  A tile's scales are whole 512-byte atoms, gathered in shared memory
// and stored 16 bytes at a time, as are the transposed codes (64 bytes a
// column).
#include <cuda.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "fp4_common.cuh"
#include "fp4_internal.h"

namespace fp8q {
namespace fp4 {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;

// Eight consecutive elements of a row as fp32.  VEC: 16-byte loads (the base
// and every row are 16-byte aligned); elements at or past `valid` read as 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int valid, float (&v)[8]) {
  if (VEC && valid >= 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
      const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < valid ? (float)p[j] : 0.0f;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int KIND, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs p) {
  constexpr int kBlock = Kind<KIND>::kBlock;
  constexpr int kAtoms = kTile / Kind<KIND>::kAtomK;   // atoms along K per tile: 1 or 2
  constexpr int kLanes = kBlock / 8;                   // lanes that share a block: 4 or 2
  __shared__ __align__(16) uint8_t s_scale[kAtoms * 512], t_scale[kAtoms * 512];
  __shared__ __align__(16) uint32_t t_code[kTile][kTile / 8 + 4];   // [column][8 rows a word]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tr = (warp >> 1) * 32 + (lane >> 3) * 8;   // this thread's first row in the tile
  const int tc = (warp & 1) * 64 + (lane & 7) * 8;     // and first column
  const unsigned tiles_c = (unsigned)((p.cols + kTile - 1) / kTile);
  const unsigned by = blockIdx.x / tiles_c, bx = blockIdx.x - by * tiles_c;
  const int64_t r0 = (int64_t)by * kTile, c0 = (int64_t)bx * kTile;
  const int64_t row = r0 + tr, col = c0 + tc;
  const T *x = static_cast<const T *>(p.x);

  float v[8][8];
  const int valid = (int)max((int64_t)0, min((int64_t)8, p.cols - col));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = row + i < p.rows && valid > 0;
    load8<T, VEC>(x + (in ? (row + i) * p.ld + col : 0), in ? valid : 0, v[i]);
  }
  const float g = KIND == FP4Q_NVFP4 ? nv_global(*p.amax) : 1.0f;
  if (KIND == FP4Q_NVFP4 && p.global_scale != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    *p.global_scale = g;

  if (p.q != nullptr) {
    const int64_t ldq = row_bytes(p.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const BlockScale b = block_scale<KIND>(m, g);
      const uint32_t w = encode8<KIND>(v[i], b);
      if (row + i < p.rows && col / 2 < ldq)
        *reinterpret_cast<uint32_t *>(p.q + (row + i) * ldq + col / 2) = w;
      if ((lane & (kLanes - 1)) == 0)
        s_scale[atom_byte(tr + i, tc / kBlock, kAtoms)] =
            (uint8_t)(row + i < p.rows && col < p.cols ? b.byte : 0u);
    }
  }
  if (p.qt != nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][j]));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8 * o));
      const BlockScale b = block_scale<KIND>(m, g);
      const float t[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
      t_code[tc + j][tr / 8] = encode8<KIND>(t, b);
      if (((lane >> 3) & (kLanes - 1)) == 0)
        t_scale[atom_byte(tc + j, tr / kBlock, kAtoms)] =
            (uint8_t)(row < p.rows && col + j < p.cols ? b.byte : 0u);
    }
  }
  __syncthreads();
  // Atoms of this tile: kAtoms consecutive ones of row block `by` (or
  // of the transpose's row block `bx`); the last tile may have fewer.
  if (threadIdx.x < kAtoms * 32) {
    const int a = threadIdx.x >> 5;
    if (p.q != nullptr) {
      const int64_t nk = num_atoms_k(KIND, p.cols), k = (int64_t)bx * kAtoms + a;
      if (k < nk)
        reinterpret_cast<uint4 *>(p.q_scales + ((int64_t)by * nk + k) * 512)[lane] =
            reinterpret_cast<const uint4 *>(s_scale + a * 512)[lane];
    }
    if (p.qt != nullptr) {
      const int64_t nk = num_atoms_k(KIND, p.rows), k = (int64_t)by * kAtoms + a;
      if (k < nk)
        reinterpret_cast<uint4 *>(p.qt_scales + ((int64_t)bx * nk + k) * 512)[lane] =
            reinterpret_cast<const uint4 *>(t_scale + a * 512)[lane];
    }
  }
  if (p.qt != nullptr) {
    const int64_t ldt = row_bytes(p.rows);
#pragma unroll
    for (int n = threadIdx.x; n < kTile * 4; n += kThreads) {   // 16-byte pieces, 32 rows each
      const int c = n >> 2, piece = n & 3;
      const int64_t at = r0 / 2 + piece * 16;
      if (c0 + c < p.cols && at < ldt)
        *reinterpret_cast<uint4 *>(p.qt + (c0 + c) * ldt + at) =
            *reinterpret_cast<const uint4 *>(&t_code[c][piece * 4]);
    }
  }
}

__global__ void global_kernel(const float *amax, float *global_scale) {
  *global_scale = nv_global(*amax);
}

// max |x| for matrices whose rows lie apart or are not 16-byte aligned.  The
// maximum of bit patterns does not depend on the order of the atomics; NaN
// patterns sort above infinity.
template <typename T>
__global__ void __launch_bounds__(256)
    amax_ld_kernel(const T *x, int64_t rows, int64_t cols, int64_t ld, unsigned int *amax) {
  uint32_t m = 0;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < cols; c += (int64_t)gridDim.x * 256)
      m = max(m, abs_bits((float)x[r * ld + c]));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __shared__ uint32_t part[8];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) m = max(m, part[i]);
    if (m != 0) atomicMax(amax, m);
  }
}

// Values of an operand: one thread per 8 codes (one 32-bit word) of a row.
template <int KIND, typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const fp4q_operand op, int64_t rows, int64_t K, T *y) {
  const int64_t ldq = row_bytes(K), words = (K + 7) / 8, nk = num_atoms_k(KIND, K);
  const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (w >= words) return;
  const float g = KIND == FP4Q_NVFP4 ? *op.global_scale : 1.0f;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint32_t code = *reinterpret_cast<const uint32_t *>(op.data + r * ldq + w * 4);
    const float s =
        scale_value<KIND>(op.scales[atom_byte(r, w * 8 / Kind<KIND>::kBlock, nk)], g);
    T *out = y + r * K + w * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w * 8 + j < K) out[j] = (T)__fmul_rn(e2m1_value(code >> (4 * j)), s);
  }
}

template <int KIND, typename T>
cudaError_t run_quantize(const QuantArgs &a, cudaStream_t stream) {
  const int64_t tiles = ((a.cols + kTile - 1) / kTile) * ((a.rows + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)tiles;
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld * (int64_t)sizeof(T) % 16 == 0;
  if (vec)
    quantize_kernel<KIND, T, true><<<grid, kThreads, 0, stream>>>(a);
  else
    quantize_kernel<KIND, T, false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(int kind, int in_dtype, const QuantArgs &a, cudaStream_t stream) {
  if (kind == FP4Q_MXFP4)
    return in_dtype == FP8Q_DT_BF16 ? run_quantize<FP4Q_MXFP4, __nv_bfloat16>(a, stream)
                                    : run_quantize<FP4Q_MXFP4, float>(a, stream);
  return in_dtype == FP8Q_DT_BF16 ? run_quantize<FP4Q_NVFP4, __nv_bfloat16>(a, stream)
                                  : run_quantize<FP4Q_NVFP4, float>(a, stream);
}

cudaError_t launch_global(const float *amax, float *global_scale, cudaStream_t stream) {
  global_kernel<<<1, 1, 0, stream>>>(amax, global_scale);
  return cudaGetLastError();
}

cudaError_t launch_amax_ld(const void *x, int in_dtype, int64_t rows, int64_t cols, int64_t ld,
                           float *amax, cudaStream_t stream) {
  if ((ld == cols || rows <= 1) && (reinterpret_cast<uintptr_t>(x) & 15u) == 0)
    return launch_amax(x, in_dtype, rows * cols, amax, stream);
  cudaError_t e = cudaMemsetAsync(amax, 0, sizeof(float), stream);
  if (e != cudaSuccess || rows * cols == 0) return e;
  const int64_t gx = std::min<int64_t>((cols + 255) / 256, 8);
  const dim3 grid((unsigned)gx, (unsigned)std::min<int64_t>(rows, 8 * sm_count() / gx + 1));
  if (in_dtype == FP8Q_DT_BF16)
    amax_ld_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16 *>(x), rows, cols, ld,
                                             reinterpret_cast<unsigned int *>(amax));
  else
    amax_ld_kernel<<<grid, 256, 0, stream>>>(static_cast<const float *>(x), rows, cols, ld,
                                             reinterpret_cast<unsigned int *>(amax));
  return cudaGetLastError();
}

cudaError_t launch_dequantize(int kind, const fp4q_operand &op, int64_t rows, int64_t K,
                              int out_dtype, void *y, cudaStream_t stream) {
  const dim3 grid((unsigned)(((K + 7) / 8 + 255) / 256), (unsigned)std::min<int64_t>(rows, 65535));
  if (kind == FP4Q_MXFP4) {
    if (out_dtype == FP8Q_DT_BF16)
      dequantize_kernel<FP4Q_MXFP4><<<grid, 256, 0, stream>>>(op, rows, K, (__nv_bfloat16 *)y);
    else
      dequantize_kernel<FP4Q_MXFP4><<<grid, 256, 0, stream>>>(op, rows, K, (float *)y);
  } else {
    if (out_dtype == FP8Q_DT_BF16)
      dequantize_kernel<FP4Q_NVFP4><<<grid, 256, 0, stream>>>(op, rows, K, (__nv_bfloat16 *)y);
    else
      dequantize_kernel<FP4Q_NVFP4><<<grid, 256, 0, stream>>>(op, rows, K, (float *)y);
  }
  return cudaGetLastError();
}

}  // namespace fp4
}  // namespace fp8q
