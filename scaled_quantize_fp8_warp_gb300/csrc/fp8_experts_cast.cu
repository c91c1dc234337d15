// The MXFP8 cast of rows in groups: rows gathered by index, 32 elements to an
// E8M0 scale 2^(floor(log2 amax) - emax), along rows and down the columns of a
// group, from one read (include/fp8q.h, fp8_quantize_experts).
//
// A block of 256 threads casts 128 rows of one group x 128 columns at a time.  A
// warp has a 32 x 32 piece, four rows x eight columns a thread, so both kinds of
// blocks of 32 lie inside a warp: maxima along a row are two shuffles away, down
// a column three.  The transposed bytes and the scales pass through shared
// memory, to leave as whole lines and atoms.
//
// What bounds it: its instructions (950 a warp and 32 x 64 elements in bf16, both
// orientations; the integer pipe is busy 53% of the time and a third of the warps
// an SM could hold are there, for want of registers), then HBM.  16384 routed rows
// of 8192 tokens x 4096 bf16 in 32 groups: 55.8 us both ways (205 MB with each token
// read once, 272 as the gather reads them: 4.9 TB/s), 35.4 by rows alone; 16384 rows
// in one group 53.0; fp32 in 32 groups 73, in 128 groups 91 (128 rows
// a group on average, most in a block that is not full or in two).  Without an index, where each row is read once, 65536 x 4096 of
// weights in 32 groups: fp32 188 by rows and 250 both ways (7.2 and 6.5 TB/s), bf16 122
// and 189 (6.6, 5.8).  In bf16 8 bytes (rows alone) or 16 (both ways) a thread spill at
// three blocks an SM, in rows that start anywhere up to 148.  70 us before the groups were found 32 at a
// time, the transposed bytes left as lines and the scales were found two at a
// time.  The next tile's loads ahead of this one's arithmetic: no gain.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp8_experts.h"
#include "fp8_pack8.cuh"

namespace fp8q {
namespace experts {
namespace {

using pack8::Pack8;

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xFFFFFFFFu;

// A block's scale X is 2^(exponent of its max |x| less the format's largest:
// 448 = 1.75 * 2^8, 57344 = 1.75 * 2^15), not below 2^-127.  Its E8M0 code from
// the maximum's biased exponent, 0xFF (NaN) for a NaN or an infinity:
template <int FMT>
__device__ __forceinline__ uint32_t scale_code(int e) {
  return e == 255 ? 0xFFu : (uint32_t)max(e - (FMT == FP8Q_E4M3 ? 8 : 15), 0);
}
// and 1 / X by the exponent's bits alone (some finite number for a NaN's), at
// the top of a 32-bit or of each 16-bit half of a word.
template <int FMT>
__device__ __forceinline__ float reciprocal(uint32_t amax_bits) {
  constexpr uint32_t kTop = (254u + (FMT == FP8Q_E4M3 ? 8u : 15u)) << 23;
  return __uint_as_float(min(kTop - (amax_bits & 0x7F800000u), 254u << 23));
}
template <int FMT>
__device__ __forceinline__ float2 reciprocals(uint32_t halves) {
  constexpr uint32_t kTop = (254u + (FMT == FP8Q_E4M3 ? 8u : 15u)) << 7;
  const uint32_t r = __vminu2(kTop * 0x10001u - (halves & 0x7F807F80u), 0x7F007F00u);
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
}
// Whether either half is an infinity's or a NaN's.
__device__ __forceinline__ bool halves_special(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Four values to bytes, saturating, the first lowest.  (Through the casting
// functions' 16-bit results every pair cost two more instructions.)
template <int FMT>
__device__ __forceinline__ uint32_t cast4(float a, float b, float c, float d) {
  uint32_t w;
  if (FMT == FP8Q_E4M3)
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}" : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}" : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// The group that block b of the operand belongs to: the last whose first block
// is not behind b.  A warp tries 32 groups at a time, so two rounds do.
__device__ __forceinline__ int group_of(const Groups &g, int b) {
  if (g.offsets == nullptr) return b / ((g.each + 127) / 128);
  int lo = 0, n = g.count;
  while (n > 1) {
    const int step = (n + 31) / 32, e = lo + (int)(threadIdx.x & 31) * step;
    const bool at = e < lo + n && first_block(g, e, min(max(g.offsets[e], 0), g.rows)) <= b;
    const int last = max(__popc(__ballot_sync(kAll, at)), 1) - 1;
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

// The scales of a 32 x 32 piece along its rows, by this thread's share of them:
// 1 / X of its four rows; find() tells whether a block of the warp holds a NaN or
// an infinity, and poison() makes those NaN.
template <int FMT, typename T>
struct RowScales;
template <int FMT>
struct RowScales<FMT, __nv_bfloat16> {
  uint32_t w[2];   // two rows' maxima each
  float f[4];
  __device__ __forceinline__ bool find(const Pack8<__nv_bfloat16> (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Pack8<__nv_bfloat16> &a = x[2 * i], &b = x[2 * i + 1];
      w[i] = __byte_perm(a.amax_bits(), b.amax_bits(), 0x7632);
      w[i] = __vmaxu2(w[i], __shfl_xor_sync(kAll, w[i], 1));
      w[i] = __vmaxu2(w[i], __shfl_xor_sync(kAll, w[i], 2));
      const float2 r = reciprocals<FMT>(w[i]);
      f[2 * i] = r.x, f[2 * i + 1] = r.y;
    }
    return __any_sync(kAll, halves_special(__vmaxu2(w[0], w[1])));
  }
  __device__ __forceinline__ void poison() {
    __syncwarp();   // a branch, not predicates on every path
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = exponent(i) == 255 ? __uint_as_float(0x7FC00000u) : f[i];
  }
  __device__ __forceinline__ int exponent(int row) const {
    return (int)((row & 2 ? w[1] : w[0]) >> (row & 1 ? 23 : 7) & 0xFFu);
  }
};
template <int FMT>
struct RowScales<FMT, float> {
  uint32_t m[4];
  float f[4];
  __device__ __forceinline__ bool find(const Pack8<float> (&x)[4]) {
    uint32_t all = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = x[i].amax_bits();
      m[i] = max(m[i], __shfl_xor_sync(kAll, m[i], 1));
      m[i] = max(m[i], __shfl_xor_sync(kAll, m[i], 2));
      f[i] = reciprocal<FMT>(m[i]);
      all = max(all, m[i]);
    }
    return __any_sync(kAll, all >= 0x7F800000u);
  }
  __device__ __forceinline__ void poison() {
    __syncwarp();   // a branch, not predicates on every path
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = exponent(i) == 255 ? __uint_as_float(0x7FC00000u) : f[i];
  }
  __device__ __forceinline__ int exponent(int row) const {
    return (int)((row & 2 ? (row & 1 ? m[3] : m[2]) : (row & 1 ? m[1] : m[0])) >> 23);
  }
};

// The same down its columns, pairs of neighbours for this thread's eight.
template <int FMT, typename T>
struct ColumnScales;
template <int FMT>
struct ColumnScales<FMT, __nv_bfloat16> {
  uint32_t w[4];
  float2 f[4];
  __device__ __forceinline__ bool find(const Pack8<__nv_bfloat16> (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = pack8::max_abs2(pack8::max_abs2(x[0].w[k], x[1].w[k]),
                             pack8::max_abs2(x[2].w[k], x[3].w[k])) & 0x7FFF7FFFu;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) w[k] = __vmaxu2(w[k], __shfl_xor_sync(kAll, w[k], o));
      f[k] = reciprocals<FMT>(w[k]);
    }
    return __any_sync(kAll, halves_special(__vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]))));
  }
  __device__ __forceinline__ void poison() {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k].x = exponent(2 * k) == 255 ? __uint_as_float(0x7FC00000u) : f[k].x;
      f[k].y = exponent(2 * k + 1) == 255 ? __uint_as_float(0x7FC00000u) : f[k].y;
    }
  }
  __device__ __forceinline__ int exponent(int column) const {
    const uint32_t v = column & 4 ? (column & 2 ? w[3] : w[2]) : (column & 2 ? w[1] : w[0]);
    return (int)(v >> (column & 1 ? 23 : 7) & 0xFFu);
  }
};
template <int FMT>
struct ColumnScales<FMT, float> {
  uint32_t m[8];
  float2 f[4];
  __device__ __forceinline__ bool find(const Pack8<float> (&x)[4]) {
    uint32_t all = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) m[j] = max(m[j], __float_as_uint(x[i].v[j]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m[j] = max(m[j], __shfl_xor_sync(kAll, m[j], o));
      all = max(all, m[j]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[k] = make_float2(reciprocal<FMT>(m[2 * k]), reciprocal<FMT>(m[2 * k + 1]));
    return __any_sync(kAll, all >= 0x7F800000u);
  }
  __device__ __forceinline__ void poison() {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k].x = exponent(2 * k) == 255 ? __uint_as_float(0x7FC00000u) : f[k].x;
      f[k].y = exponent(2 * k + 1) == 255 ? __uint_as_float(0x7FC00000u) : f[k].y;
    }
  }
  __device__ __forceinline__ int exponent(int column) const {
    uint32_t v = m[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) v = column == j ? m[j] : v;
    return (int)(v >> 23);
  }
};

// WHICH: 1 by rows, 2 transposed, 3 both.  A CTA casts `run` tiles of one block,
// one after the other.
template <int FMT, typename T, bool VEC, int WHICH>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) cast_kernel(const CastArgs p, int run) {
  __shared__ __align__(16) uint8_t atoms[2][2][512];   // of the rows, of the columns; tiles in turn
  // The columns' bytes, 128 of each column, so that they leave as whole lines;
  // words of a column are turned about by its eight's number, against bank conflicts.
  __shared__ __align__(16) uint32_t turned[WHICH & 2 ? 2 : 1][WHICH & 2 ? 128 : 1][32];
  follow_previous();
  allow_next();
  const int tiles = (p.cols + 127) / 128, runs = (tiles + run - 1) / run;
  const int block = (int)(blockIdx.x / (unsigned)runs), tile0 = (int)(blockIdx.x % (unsigned)runs) * run;
  const int tile1 = min(tile0 + run, tiles);
  const int e = group_of(p.groups, block);
  const int2 group = group_rows(p.groups, e);
  const int row0 = (block - first_block(p.groups, e, group.x)) * 128;   // in the group
  if (row0 < 0 || row0 >= group.y) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = warp >> 2;
  const int rg = lane >> 2, cg = lane & 3;
  const int r = row0 + 32 * quarter + 4 * rg;   // this thread's first row in the group
  const int left = group.y - r;                 // rows from there on
  const bool none = row0 + 32 * quarter >= group.y;   // for the whole warp
  const int col0 = 64 * half + 8 * cg;          // its first column in a tile; 32 on in step 1
  const T *from[4];
  uint32_t on = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int src = group.x + r + i;
    if (p.index != nullptr && i < left) src = p.index[src];
    const bool there = i < left && (uint32_t)src < (uint32_t)p.T;
    from[i] = static_cast<const T *>(p.x) + (int64_t)(there ? src : 0) * p.ld;
    on |= (uint32_t)there << i;
  }
  uint8_t *const q = p.q + (int64_t)(group.x + r) * p.cols;
  uint8_t *const q_t = p.q_t + 128 * (int64_t)block;
  const int64_t pitch = 128 * (int64_t)p.blocks;

  const auto load = [&](Pack8<T> (&to)[2][4], int tile) {
    const int col = 128 * tile + col0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool in = col + 32 * s < p.cols;   // all eight or none: cols % 16 == 0
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pack8::load<VEC>(to[s][i], from[i] + (in ? col + 32 * s : 0), in && (on >> i & 1) ? 8 : 0);
    }
  };
  const auto cast = [&](const Pack8<T> (&x)[2][4], int tile, int turn) {
    const int col = 128 * tile + col0;
    uint8_t (*const scale)[512] = atoms[turn];
    if (none) {   // pieces behind the group: zeros with code 0
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        scale[0][(4 * rg + cg) * 16 + quarter * 4 + 2 * half + s] = 0;
        if (!(WHICH & 2)) continue;
        scale[1][(8 * cg + rg) * 16 + (2 * half + s) * 4 + quarter] = 0;
        for (int j = 0; j < 8; ++j)
          turned[WHICH & 2 ? turn : 0][WHICH & 2 ? col0 + 32 * s + j : 0][(8 * quarter + rg) ^ (8 * cg)] = 0u;
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        RowScales<FMT, T> rows;
        ColumnScales<FMT, T> columns;
        // A block with a NaN or an infinity is multiplied by NaN, whose byte is 0x7F.
        if (WHICH & 1) {
          if (rows.find(x[s])) rows.poison();
          scale[0][(4 * rg + cg) * 16 + quarter * 4 + 2 * half + s] =
              (uint8_t)scale_code<FMT>(rows.exponent(cg));
        }
        if (WHICH & 2) {
          if (columns.find(x[s])) columns.poison();
          scale[1][(8 * cg + rg) * 16 + (2 * half + s) * 4 + quarter] =
              (uint8_t)scale_code<FMT>(columns.exponent(rg));
        }
        uint32_t *const to =
            &turned[WHICH & 2 ? turn : 0][WHICH & 2 ? col0 + 32 * s : 0][(8 * quarter + rg) ^ (8 * cg)];
        uint32_t bytes[4][2];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {   // two pairs of columns
          float2 v[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i][0] = x[s][i].pair(k), v[i][1] = x[s][i].pair(k + 1);
          if (WHICH & 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = make_float2(rows.f[i], rows.f[i]);   // powers of two: exact products
              const float2 a = __fmul2_rn(v[i][0], f), b = __fmul2_rn(v[i][1], f);
              bytes[i][k / 2] = cast4<FMT>(a.x, a.y, b.x, b.y);
            }
          }
          if (WHICH & 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 c[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) c[i] = __fmul2_rn(v[i][h], columns.f[k + h]);
              const int j = 2 * (k + h);
              to[32 * j] = cast4<FMT>(c[0].x, c[1].x, c[2].x, c[3].x);
              to[32 * (j + 1)] = cast4<FMT>(c[0].y, c[1].y, c[2].y, c[3].y);
            }
          }
        }
        if ((WHICH & 1) && col + 32 * s < p.cols) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < left)
              *reinterpret_cast<uint2 *>(q + (int64_t)i * p.cols + col + 32 * s) =
                  make_uint2(bytes[i][0], bytes[i][1]);
        }
      }
    }
    __syncthreads();   // with two turns, the one barrier of a tile
    if ((WHICH & 1) && warp == 0)
      reinterpret_cast<uint4 *>(p.q_scales + ((int64_t)block * tiles + tile) * 512)[lane] =
          reinterpret_cast<const uint4 *>(scale[0])[lane];
    if (!(WHICH & 2)) return;
    if (warp == 1)
      reinterpret_cast<uint4 *>(p.qt_scales + ((int64_t)tile * p.blocks + block) * 512)[lane] =
          reinterpret_cast<const uint4 *>(scale[1])[lane];
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // eight lanes a column
      const int c = 32 * k + threadIdx.x / 8, part = threadIdx.x & 7;
      if (128 * tile + c < p.cols)
        *reinterpret_cast<uint4 *>(q_t + (128 * tile + c) * pitch + 16 * part) =
            *reinterpret_cast<const uint4 *>(
                &turned[WHICH & 2 ? turn : 0][WHICH & 2 ? c : 0][(4 * part) ^ (8 * (c >> 3 & 3))]);
    }
  };

  for (int tile = tile0; tile < tile1; ++tile) {
    Pack8<T> x[2][4];
    load(x, tile);
    cast(x, tile, (tile - tile0) & 1);
  }
}

template <int FMT, typename T>
cudaError_t run_cast(const CastArgs &a, bool vec, cudaStream_t stream) {
  // Two tiles a CTA where that leaves the SMs work for some turns: finding the
  // group and the rows costs every CTA once (16384 rows x 4096 in 32 groups, one, two
  // and four tiles: 56.4, 54.0 and 54.6 us; 4096 rows in 64 groups: 25.6, 25.0 and 30.2).
  const int64_t tiles = (a.cols + 127) / 128;
  const int run = (int)std::min<int64_t>(2, std::max<int64_t>(1, a.blocks * tiles / (4 * sm_count())));
  const int64_t grid = a.blocks * ((tiles + run - 1) / run);
  log_line("launch experts cast_kernel %s%s, %d tiles of 128 x 128 a block, grid %lld",
           sizeof(T) == 2 ? "bf16" : "fp32", vec ? "" : " element by element", run, (long long)grid);
  Launch l((unsigned)grid, 1, kThreads, 0, stream);
  if (a.q_t == nullptr)
    return vec ? l.run(cast_kernel<FMT, T, true, 1>, a, run) : l.run(cast_kernel<FMT, T, false, 1>, a, run);
  if (a.q == nullptr)
    return vec ? l.run(cast_kernel<FMT, T, true, 2>, a, run) : l.run(cast_kernel<FMT, T, false, 2>, a, run);
  return vec ? l.run(cast_kernel<FMT, T, true, 3>, a, run) : l.run(cast_kernel<FMT, T, false, 3>, a, run);
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
