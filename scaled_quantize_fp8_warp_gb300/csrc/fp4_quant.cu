// 4-bit quantisation (MXFP4, NVFP4) and its inverse.
//
// quantize_kernel: CTAs of 256 threads own 128 x 128 tiles of x.  In one, warp w
// holds rows [32 (w / 2), +32) and columns [64 (w % 2), +64); lane l the rows
// [8 (l / 8), +8) and columns [8 (l % 8), +8) of that, so a block of 32 (or
// 16) along a row lies in 4 (2) neighbouring lanes and a block of 32 (16) down
// a column in 4 (2) lanes eight apart: both maxima are butterflies inside the
// warp.  One read of x serves both orientations; each is cast with its own
// scales.  A tile's scales are whole 512-byte atoms, gathered in shared memory
// and stored 16 bytes at a time, as are the transposed codes (64 bytes a
// column).
//
// What bounds it: neither HBM (31% busy) nor the issue slots (66% used, 20.7
// instructions an element for NVFP4 in both orientations) alone, but the three
// turns of a CTA: it loads its tile, casts all of it, then stores, with nothing
// of another tile under way, and a third of the warps an SM could hold to fill
// in.  With the encoding taken out 25.0 of 28.8 us are left.
// 8192 x 4096 bf16, both orientations: NVFP4 28.8 us (3.6 TB/s), MXFP4 26.0 us
// (4.0); 15872 x 4096, rows only: 33.7 us (4.9) and 31.2 us (5.3), of which 28.5
// and 27.4 us are left with the encoding taken out.  Three CTAs an SM: two take
// 32.2 us where three take 28.8, four 30.6 (MXFP4: 29.8, 26.0, 26.0).
#include <cuda.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fp4_common.cuh"
#include "fp4_internal.h"
#include "fp4_launch.cuh"
#include "fp8_pack8.cuh"

namespace fp8q {
namespace fp4 {
namespace {

using pack8::Pack8;
using pack8::load;

constexpr int kTile = 128;
constexpr int kThreads = 256;

// Maxima (fp32 bit patterns) of the blocks that this thread's 8 rows (m) and
// 8 columns of an 8 x 8 patch belong to: `lanes` neighbouring lanes share a
// block of a row, `lanes` lanes eight apart one of a column.  bf16 works on
// two 16-bit magnitudes to a register.
template <int LANES>
__device__ __forceinline__ void block_max_rows(const Pack8<__nv_bfloat16> (&x)[8], uint32_t (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    // high halves: rows i and i + 1
    uint32_t t = __byte_perm(x[i].amax_bits(), x[i + 1].amax_bits(), 0x7632);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) t = __vmaxu2(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
    m[i] = t << 16;
    m[i + 1] = t & 0xFFFF0000u;
  }
}

template <int LANES>
__device__ __forceinline__ void block_max_rows(const Pack8<float> (&x)[8], uint32_t (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = x[i].amax_bits();
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
  }
}

template <int LANES>
__device__ __forceinline__ void block_max_cols(const Pack8<__nv_bfloat16> (&x)[8], uint32_t (&m)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t t = x[0].w[k];
#pragma unroll
    for (int i = 1; i < 8; ++i) t = pack8::max_abs2(t, x[i].w[k]);
    t &= 0x7FFF7FFFu;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) t = __vmaxu2(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8 * o));
    m[2 * k] = t << 16;
    m[2 * k + 1] = t & 0xFFFF0000u;
  }
}

template <int LANES>
__device__ __forceinline__ void block_max_cols(const Pack8<float> (&x)[8], uint32_t (&m)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m[j] = max(m[j], __float_as_uint(x[i].v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 8 * o));
  }
}

// The transposed codes of a tile in shared memory: word w (8 rows) of column
// c.  Sixteen-byte chunks are permuted by the column and neighbouring columns
// change places in every second 32, so that a warp's stores (8 columns eight
// apart x 4 words) fall into 32 banks.
__device__ __forceinline__ int t_word(int c, int w) {
  return (c ^ ((c >> 5) & 1)) * 16 + ((((w >> 2) ^ (c >> 3)) & 3) << 2 | (w & 3));
}

// Scale bytes of eight blocks of one thread, rows (or columns) 0-3 in the low
// word.  MXFP4: from the exponents.  NVFP4: the two lanes that share the
// blocks (`mate` apart; `second` is the one with the bit set) find four each
// and swap them.
template <int KIND>
__device__ __forceinline__ void scale_bytes(const uint32_t (&m)[8], float g, float rg, int mate,
                                            bool second, uint32_t (&byte)[2]) {
  if (KIND == FP4Q_MXFP4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      byte[h] = __byte_perm(__byte_perm(mx_byte(m[4 * h]), mx_byte(m[4 * h + 1]), 0x0040),
                            __byte_perm(mx_byte(m[4 * h + 2]), mx_byte(m[4 * h + 3]), 0x0040), 0x5410);
  } else {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      t[k] = fmaxf(nv_ratio(__uint_as_float(second ? m[k + 4] : m[k]), g, rg), 0x1p-9f);
    const uint32_t mine =
        (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3) |
        (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3) << 16;
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, mine, mate);
    byte[0] = second ? other : mine;
    byte[1] = second ? mine : other;
  }
}

template <int KIND>
__device__ __forceinline__ uint32_t encode_block(const float2 (&y)[4], uint32_t byte,
                                                 const ScaleTable &table) {
  if (KIND == FP4Q_MXFP4) return encode8<KIND>(y, 0.0f, mx_reciprocal(byte));
  const float2 dr = table.d_r[byte];
  return encode8<KIND>(y, dr.x, dr.y);
}

// A tile of x in shared memory, each thread's 8 x 8 patch in 16-byte slots:
// slot (row i of the patch, 16-byte part h) of thread t at
// ((i * kParts + h) * kThreads + t) * 16.
template <typename T>
struct InTile {
  static constexpr int kParts = (int)sizeof(T) / 2;
  uint8_t at[8 * kParts * kThreads * 16];
};
struct NoTile {};

template <int KIND, typename T, bool VEC>
struct QuantSmem {
  static constexpr int kAtoms = kTile / Kind<KIND>::kAtomK;
  typename std::conditional<VEC, NoTile, InTile<T>>::type in;
  __align__(16) uint32_t t_code[kTile * 16];
  __align__(16) uint8_t s_scale[kAtoms * 512];
  __align__(16) uint8_t t_scale[kAtoms * 512];
  ScaleTable table;
};

// Rows that are not 16-byte aligned: a warp loads its 32 x 64 elements of the
// tile one by one, neighbouring lanes neighbouring elements, and deals them
// out to the lanes whose patches they belong to.
template <typename T>
__device__ __forceinline__ void load_dealt(const QuantArgs &p, int64_t row, int64_t col,
                                           InTile<T> &in, Pack8<T> (&y)[8]) {
  constexpr int kParts = InTile<T>::kParts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T *x = static_cast<const T *>(p.x);
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 8) {
    T v[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t r = row + r0 + i, c = col + lane + 32 * k;
        v[i][k] = r < p.rows && c < p.cols ? x[r * p.ld + c] : (T)0.0f;
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // element (r, c) of the 32 x 64 belongs to lane (r / 8) * 8 + c / 8
        const int c = lane + 32 * k, owner = warp * 32 + r0 + (c >> 3);
        const int byte = (c & 7) * (int)sizeof(T);
        *reinterpret_cast<T *>(in.at + ((i * kParts + (byte >> 4)) * kThreads + owner) * 16 +
                               (byte & 15)) = v[i][k];
      }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      y[i].take(h, *reinterpret_cast<const uint4 *>(
                       in.at + ((i * kParts + h) * kThreads + threadIdx.x) * 16));
}

// The matrices of one launch, their tiles numbered one matrix after the other.
// A launch of one (GROUPED false) reads it at constant offsets.
template <bool GROUPED>
struct QuantGroup {
  int n;
  unsigned tile_end[GROUPED ? kGroupMax : 1];
  QuantArgs prob[GROUPED ? kGroupMax : 1];
};

template <int KIND, typename T, bool VEC, bool GROUPED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
    quantize_kernel(const __grid_constant__ QuantGroup<GROUPED> group) {
  int which = 0;
  unsigned tile = blockIdx.x;
  if (GROUPED) {
    while (which + 1 < group.n && blockIdx.x >= group.tile_end[which]) ++which;
    if (which > 0) tile -= group.tile_end[which - 1];
  }
  const QuantArgs &p = group.prob[which];
  constexpr int kBlock = Kind<KIND>::kBlock;
  constexpr int kAtoms = kTile / Kind<KIND>::kAtomK;   // atoms along K per tile: 1 or 2
  constexpr int kLanes = kBlock / 8;                   // lanes that share a block: 4 or 2
  extern __shared__ __align__(16) uint8_t smem[];
  auto &sm = *reinterpret_cast<QuantSmem<KIND, T, VEC> *>(smem);
  uint8_t *const s_scale = sm.s_scale, *const t_scale = sm.t_scale;
  uint32_t *const t_code = sm.t_code;
  ScaleTable &table = sm.table;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tr = (warp >> 1) * 32 + (lane >> 3) * 8;   // this thread's first row in the tile
  const int tc = (warp & 1) * 64 + (lane & 7) * 8;     // and first column
  const unsigned tiles_c = (unsigned)((p.cols + kTile - 1) / kTile);
  const unsigned by = tile / tiles_c, bx = tile - by * tiles_c;
  const int64_t r0 = (int64_t)by * kTile, c0 = (int64_t)bx * kTile;
  const int64_t row = r0 + tr, col = c0 + tc;
  const int rows_in = (int)max((int64_t)0, min((int64_t)8, p.rows - row));
  const int cols_in = (int)max((int64_t)0, min((int64_t)8, p.cols - col));

  follow_previous();
  allow_next();
  Pack8<T> y[8];
  if constexpr (VEC) {
    const T *x = static_cast<const T *>(p.x) + (rows_in > 0 && cols_in > 0 ? row * p.ld + col : 0);
    if (rows_in == 8 && cols_in == 8) {   // all loads in a row, no test between them
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i].load_vec(x + i * p.ld);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        load<true>(y[i], i < rows_in ? x + i * p.ld : x, i < rows_in ? cols_in : 0);
    }
  } else {
    load_dealt(p, r0 + (warp >> 1) * 32, c0 + (warp & 1) * 64, sm.in, y);
  }
  float g = 1.0f, rg = 1.0f;
  if (KIND == FP4Q_NVFP4) {
    g = nv_global(*p.amax);
    rg = __frcp_rn(g);
    table.fill(g);
    if (p.global_scale != nullptr && tile == 0 && threadIdx.x == 0) *p.global_scale = g;
    __syncthreads();
  }
  if (p.q != nullptr) {
    const int64_t ldq = row_bytes(p.cols);
    uint8_t *q = p.q + row * ldq + col / 2;
    if (col / 2 >= ldq) q = nullptr;
    uint8_t *scale = s_scale + atom_byte(tr, tc / kBlock, kAtoms);
    const bool first = (lane & (kLanes - 1)) == 0;
    uint32_t m[8], top = 0;
    block_max_rows<kLanes>(y, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, m[i]);
    if (!__any_sync(0xFFFFFFFFu, top >= kCarefulBits || !(g < __uint_as_float(0x7F800000u)))) {
      uint32_t byte[2];
      scale_bytes<KIND>(m, g, rg, 1, lane & 1, byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = (byte[i >> 2] >> (8 * (i & 3))) & 0xFFu;
        const float2 v[4] = {y[i].pair(0), y[i].pair(1), y[i].pair(2), y[i].pair(3)};
        const uint32_t w = encode_block<KIND>(v, b, table);
        if (i < rows_in && q != nullptr) *reinterpret_cast<uint32_t *>(q + i * ldq) = w;
        if (first) scale[16 * i] = (uint8_t)(i < rows_in && cols_in > 0 ? b : 0u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t b;
        const uint32_t w = encode8_careful<KIND>(y[i].pair(0), y[i].pair(1), y[i].pair(2),
                                                 y[i].pair(3), m[i], g, &b);
        if (i < rows_in && q != nullptr) *reinterpret_cast<uint32_t *>(q + i * ldq) = w;
        if (first) scale[16 * i] = (uint8_t)(i < rows_in && cols_in > 0 ? b : 0u);
      }
    }
  }
  if (p.qt != nullptr) {
    uint8_t *scale = t_scale + atom_byte(tc, tr / kBlock, kAtoms);
    const bool first = ((lane >> 3) & (kLanes - 1)) == 0;
    uint32_t m[8], top = 0;
    block_max_cols<kLanes>(y, m);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, m[j]);
    if (!__any_sync(0xFFFFFFFFu, top >= kCarefulBits || !(g < __uint_as_float(0x7F800000u)))) {
      uint32_t byte[2];
      scale_bytes<KIND>(m, g, rg, 8, lane & 8, byte);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = (byte[j >> 2] >> (8 * (j & 3))) & 0xFFu;
        const float2 v[4] = {make_float2(y[0].at(j), y[1].at(j)), make_float2(y[2].at(j), y[3].at(j)),
                             make_float2(y[4].at(j), y[5].at(j)), make_float2(y[6].at(j), y[7].at(j))};
        t_code[t_word(tc + j, tr / 8)] = encode_block<KIND>(v, b, table);
        if (first) scale[16 * j] = (uint8_t)(rows_in > 0 && j < cols_in ? b : 0u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t b;
        t_code[t_word(tc + j, tr / 8)] = encode8_careful<KIND>(
            make_float2(y[0].at(j), y[1].at(j)), make_float2(y[2].at(j), y[3].at(j)),
            make_float2(y[4].at(j), y[5].at(j)), make_float2(y[6].at(j), y[7].at(j)), m[j], g, &b);
        if (first) scale[16 * j] = (uint8_t)(rows_in > 0 && j < cols_in ? b : 0u);
      }
    }
  }
  __syncthreads();
  // Atoms of this tile: kAtoms consecutive ones of row block `by` (or of the
  // transpose's row block `bx`); the last tile may have fewer.
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
            *reinterpret_cast<const uint4 *>(&t_code[t_word(c, piece * 4)]);
    }
  }
}

__global__ void global_kernel(const float *amax, float *global_scale) {
  follow_previous();
  allow_next();
  *global_scale = nv_global(*amax);
}

// max |x| of a span of a matrix, into *amax.  The maximum of bit patterns does
// not depend on the order of the atomics; NaN patterns sort above infinity.
__device__ __forceinline__ void publish_amax(uint32_t m, unsigned int *amax) {
  __shared__ uint32_t part[kThreads / 32];
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, part[i]);
    if (m != 0) atomicMax(amax, m);
  }
}

// This CTA's share of one row; VEC: the row is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t row_amax(const T *p, int64_t cols) {
  constexpr int kBatch = 4;   // groups of 8 elements in flight
  uint32_t m = 0;
  const int64_t step = (int64_t)gridDim.x * kThreads * (VEC ? 8 : 1);
  const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * (VEC ? 8 : 1);
  if (VEC) {
    for (int64_t c = first; c < cols; c += kBatch * step) {
      Pack8<T> v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int64_t left = cols - (c + b * step);
        if (left >= 8)
          v[b].load_vec(p + c + b * step);
        else
          v[b].load_some(p + (left > 0 ? c + b * step : 0), (int)max(left, (int64_t)0));
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) m = max(m, v[b].amax_bits());
    }
  } else {
    for (int64_t c = first; c < cols; c += step)
      m = max(m, __float_as_uint((float)p[c]) & 0x7FFFFFFFu);
  }
  return m;
}

// A matrix whose rows lie ld apart.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    amax_rows_kernel(const T *x, int64_t rows, int64_t cols, int64_t ld, unsigned int *amax) {
  follow_previous();
  allow_next();
  uint32_t m = 0;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    m = max(m, row_amax<T, VEC>(x + r * ld, cols));
  publish_amax(m, amax);
}

// Dense matrices, blockIdx.y of them.  The three of a training
// step's 4096-wide linear (8192 x 4096, 4096 x 4096, 8192 x 4096; 168 MB of bf16)
// take 33 us (5.0 TB/s).
struct AmaxGroup {
  const void *x[kGroupMax];
  int64_t size[kGroupMax];
};
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    amax_group_kernel(const __grid_constant__ AmaxGroup group, unsigned int *amax) {
  follow_previous();
  allow_next();
  publish_amax(row_amax<T, VEC>(static_cast<const T *>(group.x[blockIdx.y]), group.size[blockIdx.y]),
               amax + blockIdx.y);
}

// Values of an operand: one thread per 8 codes (one 32-bit word) of kRows rows
// at a time, whose reads are in flight together.  VEC: every row of y starts on
// a 16-byte boundary and K is a multiple of 16.  For fp32 two neighbouring
// lanes (16 codes, one scale) share their words out so that together they
// store whole 32-byte sectors.  Otherwise a warp's 256 values of a row pass
// through shared memory and leave one by one, neighbouring lanes neighbouring
// elements.  8192 x 4096 NVFP4 to fp32 24.3 us (6.3 TB/s, bound by the stores),
// MXFP4 to bf16 16.4 us (5.2); 1003 x 2570 to bf16 5.2 us.
template <int KIND, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const fp4q_operand op, int64_t rows, int64_t K, T *y) {
  constexpr int kRows = 4;
  constexpr bool kShare = VEC && sizeof(T) == 4;
  __shared__ __align__(16) T turn[VEC ? 1 : kThreads / 32][VEC ? 1 : 256];
  const int lane = threadIdx.x & 31;
  const int64_t ldq = row_bytes(K), nk = num_atoms_k(KIND, K);
  const int64_t w = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int valid = (int)max((int64_t)0, min((int64_t)8, K - w * 8));
  const bool odd = threadIdx.x & 1;
  follow_previous();
  allow_next();
  const float g = KIND == FP4Q_NVFP4 ? *op.global_scale : 1.0f;
  for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < rows; r0 += (int64_t)gridDim.y * kRows) {
    uint32_t code[kRows], byte[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = min(r0 + i, rows - 1);
      code[i] = byte[i] = 0u;
      if (valid > 0) {
        code[i] = *reinterpret_cast<const uint32_t *>(op.data + r * ldq + w * 4);
        byte[i] = op.scales[atom_byte(r, w * 8 / Kind<KIND>::kBlock, nk)];
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float s = scale_value<KIND>(byte[i], g);
      uint32_t c = code[i];
      if (kShare) {   // even lanes: both low halves, odd lanes: both high ones
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, c, 1);
        c = odd ? __byte_perm(other, c, 0x7632) : __byte_perm(c, other, 0x5410);
      }
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = e2m1x2_values(c >> (8 * j));
        v[2 * j] = __fmul_rn(f.x, s);
        v[2 * j + 1] = __fmul_rn(f.y, s);
      }
      T *out = y + (r0 + i) * K + w * 8;
      if constexpr (!VEC) {
        T *line = turn[threadIdx.x >> 5];
        pack8::store<true>(line + lane * 8, 8, v);
        __syncwarp();
        const int64_t c0 = (w - lane) * 8;   // the warp's first column
        if (r0 + i < rows)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c0 + lane + 32 * k < K) y[(r0 + i) * K + c0 + lane + 32 * k] = line[lane + 32 * k];
        __syncwarp();
        continue;
      }
      if (r0 + i >= rows || valid == 0) continue;
      if constexpr (kShare) {
        out += odd ? -4 : 0;
        *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(out + 8) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        pack8::store<VEC>(out, valid, v);
      }
    }
  }
}

template <int KIND, typename T, bool VEC, bool GROUPED>
cudaError_t start_quantize(const QuantArgs *a, int n, cudaStream_t stream) {
  auto kernel = quantize_kernel<KIND, T, VEC, GROUPED>;
  constexpr int smem = (int)sizeof(QuantSmem<KIND, T, VEC>);
  if (smem > 48 * 1024) {
    static PerDeviceOnce setup;   // per instantiation
    if (setup.get([&] {
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
                         cudaSuccess
                     ? 1
                     : 0;
        }) != 1)
      return cudaErrorInvalidValue;
  }
  QuantGroup<GROUPED> group{};
  group.n = n;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    tiles += ((a[i].cols + kTile - 1) / kTile) * ((a[i].rows + kTile - 1) / kTile);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    group.tile_end[i] = (unsigned)tiles;
    group.prob[i] = a[i];
  }
  log_line("launch fp4 quantize_kernel kind %d %s input%s, %d matrices, tiles of 128x128, grid %lld",
           KIND, sizeof(T) == 2 ? "bf16" : "fp32", VEC ? "" : " element by element", n,
           (long long)tiles);
  return Launch((unsigned)tiles, 1, kThreads, smem, stream).run(kernel, group);
}

template <int KIND, typename T>
cudaError_t run_quantize(const QuantArgs *a, int n, cudaStream_t stream) {
  bool vec = true;
  for (int i = 0; i < n; ++i)
    vec = vec && (reinterpret_cast<uintptr_t>(a[i].x) & 15u) == 0 &&
          a[i].ld * (int64_t)sizeof(T) % 16 == 0 && a[i].cols % 8 == 0;
  if (n == 1)
    return vec ? start_quantize<KIND, T, true, false>(a, n, stream)
               : start_quantize<KIND, T, false, false>(a, n, stream);
  return vec ? start_quantize<KIND, T, true, true>(a, n, stream)
             : start_quantize<KIND, T, false, true>(a, n, stream);
}

}  // namespace

cudaError_t launch_quantize(int kind, int in_dtype, const QuantArgs *a, int n, cudaStream_t stream) {
  if (kind == FP4Q_MXFP4)
    return in_dtype == FP8Q_DT_BF16 ? run_quantize<FP4Q_MXFP4, __nv_bfloat16>(a, n, stream)
                                    : run_quantize<FP4Q_MXFP4, float>(a, n, stream);
  return in_dtype == FP8Q_DT_BF16 ? run_quantize<FP4Q_NVFP4, __nv_bfloat16>(a, n, stream)
                                  : run_quantize<FP4Q_NVFP4, float>(a, n, stream);
}

cudaError_t launch_global(const float *amax, float *global_scale, cudaStream_t stream) {
  log_line("launch fp4 global_kernel grid 1");
  return Launch(1, 1, 1, 0, stream).run(global_kernel, amax, global_scale);
}

template <typename T>
static cudaError_t start_amax(const void *x, int64_t rows, int64_t cols, int64_t ld, unsigned int *amax,
                       cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
  // about 8 CTAs an SM, each with a batch of loads for its threads
  const int64_t per_cta = kThreads * (vec ? 8 * 4 : 8);
  const int64_t gx = std::min<int64_t>((cols + per_cta - 1) / per_cta, 8 * sm_count());
  const unsigned gy = (unsigned)std::min<int64_t>(rows, 8 * sm_count() / gx + 1);
  log_line("launch fp4 amax_rows_kernel %s input, %lldx%lld, grid %lldx%u",
           sizeof(T) == 2 ? "bf16" : "fp32", (long long)rows, (long long)cols, (long long)gx, gy);
  return Launch((unsigned)gx, gy, kThreads, 0, stream)
      .run(vec ? amax_rows_kernel<T, true> : amax_rows_kernel<T, false>, static_cast<const T *>(x), rows, cols,
           ld, amax);
}

cudaError_t launch_amax_ld(const void *x, int in_dtype, int64_t rows, int64_t cols, int64_t ld,
                           float *amax, cudaStream_t stream) {
  // a dense matrix is one long row for the per-tensor amax
  if ((ld == cols || rows <= 1) && (reinterpret_cast<uintptr_t>(x) & 15u) == 0)
    return launch_amax(x, in_dtype, rows * cols, amax, stream);
  cudaError_t e = cudaMemsetAsync(amax, 0, sizeof(float), stream);
  if (e != cudaSuccess || rows == 0 || cols == 0) return e;
  unsigned int *m = reinterpret_cast<unsigned int *>(amax);
  return in_dtype == FP8Q_DT_BF16 ? start_amax<__nv_bfloat16>(x, rows, cols, ld, m, stream)
                                  : start_amax<float>(x, rows, cols, ld, m, stream);
}

template <typename T>
static cudaError_t start_amax_group(const AmaxGroup &group, int n, unsigned int *amax,
                                    cudaStream_t stream) {
  bool vec = true;
  int64_t most = 1;
  for (int i = 0; i < n; ++i) {
    vec = vec && (reinterpret_cast<uintptr_t>(group.x[i]) & 15u) == 0;
    most = std::max(most, group.size[i]);
  }
  const int64_t per_cta = kThreads * (vec ? 8 * 4 : 8);
  const unsigned gx = (unsigned)std::min<int64_t>((most + per_cta - 1) / per_cta, 8 * sm_count() / n);
  log_line("launch fp4 amax_group_kernel %s input, grid %ux%d", sizeof(T) == 2 ? "bf16" : "fp32", gx, n);
  return Launch(gx, (unsigned)n, kThreads, 0, stream)
      .run(vec ? amax_group_kernel<T, true> : amax_group_kernel<T, false>, group, amax);
}

cudaError_t launch_amax_group(const void *const *x, const int64_t *size, int n, int in_dtype,
                              float *amax, cudaStream_t stream) {
  const cudaError_t e = cudaMemsetAsync(amax, 0, n * sizeof(float), stream);
  if (e != cudaSuccess) return e;
  AmaxGroup group{};
  for (int i = 0; i < n; ++i) group.x[i] = x[i], group.size[i] = size[i];
  unsigned int *m = reinterpret_cast<unsigned int *>(amax);
  return in_dtype == FP8Q_DT_BF16 ? start_amax_group<__nv_bfloat16>(group, n, m, stream)
                                  : start_amax_group<float>(group, n, m, stream);
}

template <int KIND, typename T>
static cudaError_t run_dequantize(const fp4q_operand &op, int64_t rows, int64_t K, void *y,
                                  cudaStream_t stream) {
  const int64_t gx = (K + 8 * kThreads - 1) / (8 * kThreads);
  if (gx > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned gy = (unsigned)std::min<int64_t>((rows + 3) / 4, 65535);
  log_line("launch fp4 dequantize_kernel kind %d %s output, four rows of 2048 columns a CTA, grid %lldx%u",
           KIND, sizeof(T) == 2 ? "bf16" : "fp32", (long long)gx, gy);
  return Launch((unsigned)gx, gy, kThreads, 0, stream)
      .run(K % 16 == 0 ? dequantize_kernel<KIND, T, true> : dequantize_kernel<KIND, T, false>, op,
           rows, K, static_cast<T *>(y));
}

cudaError_t launch_dequantize(int kind, const fp4q_operand &op, int64_t rows, int64_t K,
                              int out_dtype, void *y, cudaStream_t stream) {
  if (kind == FP4Q_MXFP4)
    return out_dtype == FP8Q_DT_BF16
               ? run_dequantize<FP4Q_MXFP4, __nv_bfloat16>(op, rows, K, y, stream)
               : run_dequantize<FP4Q_MXFP4, float>(op, rows, K, y, stream);
  return out_dtype == FP8Q_DT_BF16
             ? run_dequantize<FP4Q_NVFP4, __nv_bfloat16>(op, rows, K, y, stream)
             : run_dequantize<FP4Q_NVFP4, float>(op, rows, K, y, stream);
}

}  // namespace fp4
}  // namespace fp8q
