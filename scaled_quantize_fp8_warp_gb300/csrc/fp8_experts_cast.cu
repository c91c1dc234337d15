// The MXFP8 cast of rows in groups: rows gathered by index, 32 elements to an
// E8M0 scale 2^(floor(log2 amax) - emax), along rows and down the columns of a
// group, from one read (include/fp8q.h, fp8_quantize_experts).
//
// A block of 256 threads casts 128 rows of one group x 128 columns.  A warp
// has a 32 x 32 piece at a time, four rows x eight columns a thread, so both
// kinds of blocks of 32 lie inside a warp: maxima along a row are two shuffles
// away, down a column three, and nothing passes through shared memory but the
// scales, which leave as whole atoms.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "fp4_launch.cuh"
#include "fp8_experts.h"
#include "fp8_pack8.cuh"

namespace fp8q {
namespace experts {
namespace {

using pack8::Pack8;

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xFFFFFFFFu;

// E8M0 code of a block from its max |x|: the exponent of amax less the
// format's largest (448 = 1.75 * 2^8, 57344 = 1.75 * 2^15), not below 2^-127;
// 0xFF (NaN) where the block holds a NaN or an infinity.
template <int FMT>
__device__ __forceinline__ uint32_t scale_code(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? 0xFFu : (uint32_t)max(e - (FMT == FP8Q_E4M3 ? 8 : 15), 0);
}

// 2^(127 - code): code is at most 246 for a finite maximum.
__device__ __forceinline__ float reciprocal(uint32_t code) {
  return __uint_as_float((254u - min(code, 254u)) << 23);
}

template <int FMT>
__device__ __forceinline__ uint32_t cast2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE,
                                            FMT == FP8Q_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// Four bytes under their reciprocals (a product with a power of two: exact).
template <int FMT>
__device__ __forceinline__ uint32_t cast4(float a, float b, float c, float d, float r) {
  return __byte_perm(cast2<FMT>(a * r, b * r), cast2<FMT>(c * r, d * r), 0x5410);
}

// The group that block b of the operand belongs to.
__device__ __forceinline__ int group_of(const Groups &g, int b) {
  if (g.offsets == nullptr) return b / ((g.each + 127) / 128);
  int lo = 0, hi = g.count;   // first_block(lo) <= b < first_block(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first_block(g, mid, min(max(g.offsets[mid], 0), g.rows)) <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) cast_kernel(const CastArgs p) {
  __shared__ __align__(16) uint8_t atoms[2][512];   // of the rows, of the columns
  follow_previous();
  allow_next();
  const int tiles = (p.cols + 127) / 128;
  const int block = (int)(blockIdx.x / (unsigned)tiles), tile = (int)(blockIdx.x % (unsigned)tiles);
  const int e = group_of(p.groups, block);
  const int2 group = group_rows(p.groups, e);
  const int row0 = (block - first_block(p.groups, e, group.x)) * 128;   // in the group
  if (row0 < 0 || row0 >= group.y) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = warp >> 2;
  const int rg = lane >> 2, cg = lane & 3;
  const int r = row0 + 32 * quarter + 4 * rg;            // this thread's first row in the group
  const int col = 128 * tile + 64 * half + 8 * cg;       // and its first column; 32 on in step 1
  Pack8<T> x[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t from = -1;
    if (r + i < group.y) {
      from = group.x + r + i;
      if (p.index != nullptr) from = p.index[from];
    }
    const bool on = from >= 0 && from < p.T;
    const T *row = static_cast<const T *>(p.x) + (on ? from * p.ld : 0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int valid = on && col + 32 * s < p.cols ? 8 : 0;   // cols % 16 == 0
      pack8::load<VEC>(x[s][i], row + (valid ? col + 32 * s : 0), valid);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int c = col + 32 * s;
    if (p.q != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t m = x[s][i].amax_bits();
        m = max(m, __shfl_xor_sync(kAll, m, 1));
        m = max(m, __shfl_xor_sync(kAll, m, 2));
        const uint32_t code = scale_code<FMT>(m);
        const float f = reciprocal(code);
        const Pack8<T> &v = x[s][i];
        uint2 w = make_uint2(cast4<FMT>(v.at(0), v.at(1), v.at(2), v.at(3), f),
                             cast4<FMT>(v.at(4), v.at(5), v.at(6), v.at(7), f));
        if (code == 0xFFu) w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (cg == 0) atoms[0][(4 * rg + i) * 16 + quarter * 4 + 2 * half + s] = (uint8_t)code;
        if (r + i < group.y && c < p.cols)
          *reinterpret_cast<uint2 *>(p.q + (int64_t)(group.x + r + i) * p.cols + c) = w;
      }
    }
    if (p.q_t != nullptr) {
      uint8_t *to = p.q_t + (int64_t)c * (128 * (int64_t)p.blocks) + 128 * (int64_t)block +
                    32 * quarter + 4 * rg;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[s][i].at(j)) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
        const uint32_t code = scale_code<FMT>(m);
        uint32_t w = cast4<FMT>(x[s][0].at(j), x[s][1].at(j), x[s][2].at(j), x[s][3].at(j),
                                reciprocal(code));
        if (code == 0xFFu) w = 0x7F7F7F7Fu;
        if (rg == 0)
          atoms[1][(8 * cg + j) * 16 + (2 * half + s) * 4 + quarter] = (uint8_t)code;
        if (c < p.cols)
          *reinterpret_cast<uint32_t *>(to + j * (128 * (int64_t)p.blocks)) = w;
      }
    }
  }
  __syncthreads();
  const int t = threadIdx.x & 31;
  if (warp == 0 && p.q != nullptr)
    reinterpret_cast<uint4 *>(p.q_scales + ((int64_t)block * tiles + tile) * 512)[t] =
        reinterpret_cast<const uint4 *>(atoms[0])[t];
  if (warp == 1 && p.q_t != nullptr)
    reinterpret_cast<uint4 *>(p.qt_scales + ((int64_t)tile * p.blocks + block) * 512)[t] =
        reinterpret_cast<const uint4 *>(atoms[1])[t];
}

template <int FMT, typename T>
cudaError_t run_cast(const CastArgs &a, bool vec, cudaStream_t stream) {
  const int64_t grid = (int64_t)a.blocks * ((a.cols + 127) / 128);
  log_line("launch experts cast_kernel %s%s, 128 x 128 a block, grid %lld",
           sizeof(T) == 2 ? "bf16" : "fp32", vec ? "" : " element by element", (long long)grid);
  Launch l((unsigned)grid, 1, kThreads, 0, stream);
  return vec ? l.run(cast_kernel<FMT, T, true>, a) : l.run(cast_kernel<FMT, T, false>, a);
}

}  // namespace

cudaError_t launch_cast(int in_dtype, int format, const CastArgs &a, cudaStream_t stream) {
  const int64_t size = in_dtype == FP8Q_DT_BF16 ? 2 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld * size % 16 == 0;
  if (in_dtype == FP8Q_DT_BF16)
    return format == FP8Q_E4M3 ? run_cast<FP8Q_E4M3, __nv_bfloat16>(a, vec, stream)
                               : run_cast<FP8Q_E5M2, __nv_bfloat16>(a, vec, stream);
  return format == FP8Q_E4M3 ? run_cast<FP8Q_E4M3, float>(a, vec, stream)
                             : run_cast<FP8Q_E5M2, float>(a, vec, stream);
}

}  // namespace experts
}  // namespace fp8q
