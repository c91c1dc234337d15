// The 4-bit product for few rows: y[M, N] = x . w^T where reading w once is
// the work (M = 1: two operations per code read) or where 256 x 256 tiles
// would leave most SMs idle.
//
// The operands change places: 128 rows of w are the MMA's M, up to 128 rows of
// x its N, so that one row of x costs an MMA of N = 16 and not of 128.  The K
// range of a tile is split over the CTAs of a cluster, which stream their
// parts of w at once; their partial sums meet in distributed shared memory and
// are added in the order of the ranks, so results do not depend on timing.
// For a few rows of x in bf16 or fp32 the kernel quantises them itself, each
// CTA its own K range, while its part of w is on the way: one launch in all.
//
// Roles: warp 0 loads (TMA), warp 1 issues the MMAs, warps 2-9 quantise x and
// then add, scale and store.  Two CTAs share an SM: 256 of the 512 columns of
// tensor memory each.  (No third one fits their 112 KB of shared memory, nor any
// other kernel of this library that allocates tensor memory: an allocation
// never waits for a CTA that waits for this one's cluster.)
//
// What bounds it: latency for one row, then the casting of x, which every tile
// repeats.  In a graph, one row and 16 rows, each call with another w so that all
// come from HBM: MXFP4 1024 x 4096 4.2 and 4.7 us, 12288 x 4096 8.4 and 11.1, 4096 x
// 16384 10.1 and 12.3; NVFP4 4.8 and 5.3, 9.1 and 11.7, 10.8 and 13.0 (bytes at the
// measured copy rate: 0.3, 4 and 5.3).  With w in L2: MXFP4 4.0 and 4.7, 7.3 and
// 10.2, 8.2 and 11.0; NVFP4 4.7 and 5.3, 8.1 and 11.5, 8.8 and 12.2.  Casting x in a
// launch of its own takes from HBM 1.3-3.1 us more for one row and 1.0-1.5 us
// more for 16, but for 12288 x 4096, where 16 rows are level in NVFP4 and 0.65 us
// less in MXFP4; with w in L2 12288 x 4096 takes 1.6 us less apart at 16 rows and
// is level at nine, 4096 x 16384 is level at 13.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_common.cuh"
#include "fp4_internal.h"
#include "fp4_launch.cuh"
#include "fp4_ptx.cuh"
#include "fp8_pack8.cuh"
#include "fp8q_gemm_common.cuh"

namespace fp8q {
namespace fp4 {
namespace {

using namespace ptx;
using pack8::Pack8;

constexpr int kThreads = 320;
constexpr int kQuantWarps = 8;
constexpr int kBKBytes = 128, kBK = 256;    // K per stage
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;                // CTAs of a cluster (the portable limit)
constexpr int kMaxRows = 128;               // rows of x per tile
constexpr uint32_t kTmemCols = 256;
constexpr int kSmemBytes = 112 * 1024;      // two CTAs on an SM, never three
constexpr int kFixedBytes = 1024 /* alignment */ + 8 * (2 * kMaxStages + 2) + 16 + 1024 /* table */;

struct Args {
  int64_t M, N, K, ldx;
  const void *x;
  const float *x_amax;       // quantising NVFP4
  const float *gx, *gw;      // NVFP4 tensor scales (gx: of a quantised x)
  void *y;
  int nb;                    // rows of x per tile: 16, 32, 64 or 128
  int m_tiles, split, stages, stage_bytes;
  int num_k_blocks, num_steps, atoms_k;
  int vec, out_bf16;
  uint32_t idesc;
  unsigned int *err;
};

struct Maps {
  CUtensorMap w, sfw, x, sfx;
};

// The products of one launch, their tiles numbered one product after the
// other.  A launch of one (GROUPED false) reads it at constant offsets.
template <bool GROUPED>
struct Group {
  static constexpr int kMax = GROUPED ? kGroupMax : 1;
  int n;
  int tile_end[kMax];
  Args prob[kMax];
  Maps maps[kMax];
};

// XT: the type of x to quantise, or void for a quantised x.
template <int KIND, typename XT, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 2)
    split_kernel(const __grid_constant__ Group<GROUPED> group) {
  int which = 0, tile = blockIdx.x / group.prob[0].split;   // one split for all
  if (GROUPED) {
    while (which + 1 < group.n && tile >= group.tile_end[which]) ++which;
    if (which > 0) tile -= group.tile_end[which - 1];
  }
  const Args &p = group.prob[which];
  const Maps &maps = group.maps[which];
  constexpr int kAtoms = kBK / Kind<KIND>::kAtomK;
  constexpr bool kQuantize = !std::is_same<XT, void>::value;
  constexpr int kSfaOff = 128 * kBKBytes, kSfbOff = kSfaOff + kAtoms * 512;
  constexpr int kXOff = (kSfbOff + kAtoms * 512 + 1023) / 1024 * 1024;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t *ring_ptr = smem_raw + (ring - raw);
  const uint32_t bars = ring + p.stages * p.stage_bytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kMaxStages;
  const uint32_t accf = bars + 8 * (2 * kMaxStages), drain = accf + 8;
  uint8_t *slot_ptr = smem_raw + (drain + 8 - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);
  const uint32_t free_kb = smem_u32(slot_ptr + 8);   // K blocks below this have a free slot
  ScaleTable &table = *reinterpret_cast<ScaleTable *>(slot_ptr + 16);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.split > 1 ? cluster_ctarank() : 0u;
  const int nt = tile / p.m_tiles, mt = tile - nt * p.m_tiles;
  const int rows = (int)min((int64_t)p.nb, p.M - (int64_t)mt * p.nb);   // of x in this tile
  // K blocks of this CTA
  const int kb0 = (int)((int64_t)p.num_k_blocks * rank / p.split);
  const int kb1 = (int)((int64_t)p.num_k_blocks * (rank + 1) / p.split);
  const uint32_t sf_col0 = max(32, p.nb);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8 * s, kQuantize ? 1 + (rows + 3) / 4 : 1);   // loads; tasks
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    counter_set(free_kb, 0);
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.sfw);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(slot_ptr), kTmemCols);
    tmem_relinquish();
  }
  follow_previous();
  allow_next();
  float g = 1.0f, rg = 1.0f;
  if (kQuantize && KIND == FP4Q_NVFP4) {
    g = nv_global(*p.x_amax);
    rg = __frcp_rn(g);
    table.fill(g);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % p.stages, ph = (it / p.stages) & 1;
        const uint32_t full = full0 + 8 * s;
        if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (kQuantize) counter_set(free_kb, it + 1);
        const uint32_t sa = ring + s * p.stage_bytes;
        const int ka = kb * kAtoms;
        mbar_arrive_expect_tx(full, 128 * kBKBytes + kAtoms * 512 +
                                        (kQuantize ? 0 : p.nb * kBKBytes + kAtoms * 512));
        tma_load_2d(sa, &maps.w, kb * kBKBytes, nt * 128, full);
        // Atoms past the last of a row block are the next block's or zeros;
        // no MMA step reads them.
        tma_load_2d(sa + kSfaOff, &maps.sfw, 0, nt * p.atoms_k + ka, full);
        if (!kQuantize) {
          // more than one tile of rows only where a tile has 128
          tma_load_2d(sa + kXOff, &maps.x, kb * kBKBytes, mt * p.nb, full);
          tma_load_2d(sa + kSfbOff, &maps.sfx, 0, mt * p.atoms_k + ka, full);
        }
      }
      if (!ok) {
        // Let the copies already issued land before the CTA goes away.
        for (int j = 0; j < min(it, p.stages); ++j) {
          const int jj = it - 1 - j;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full0 + 8 * (jj % p.stages), (jj / p.stages) & 1) &&
                 globaltimer_ns() - t0 < 200000000ull) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    bool ok = true;
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % p.stages, ph = (it / p.stages) & 1;
      if (!wait_bounded_all(full0 + 8 * s, ph, abort_flag, p.err)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = ring + s * p.stage_bytes;
        const uint32_t sfa = tmem_base + sf_col0 + 8u * kAtoms * s, sfb = sfa + 4 * kAtoms;
        const uint64_t atom = sdesc_plain(sa + kSfaOff, 128);
#pragma unroll
        for (int a = 0; a < kAtoms; ++a) {
          tmem_cp_32x128b_x4(sfa + 4 * a, atom + 32 * a);
          tmem_cp_32x128b_x4(sfb + 4 * a, atom + 32 * (kAtoms + a));
        }
        const uint64_t ad = sdesc_k(sa, gemm::kSwzSBO, gemm::kSwzMode);
        const uint64_t bd = sdesc_k(sa + kXOff, gemm::kSwzSBO, gemm::kSwzMode);
        const int steps = p.num_steps - 4 * kb;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < steps) {
            const int a = KIND == FP4Q_MXFP4 ? k >> 1 : k;
            const uint32_t half = KIND == FP4Q_MXFP4 ? 2u * (k & 1) : 0u;
            mma_fp4<KIND>(tmem_base, ad + 2 * k, bd + 2 * k, p.idesc | (half << 29) | (half << 4),
                          sfa + 4 * a, sfb + 4 * a, (it > 0 || k > 0) ? 1u : 0u);
          }
        }
        mma_commit(empty0 + 8 * s);
        if (kb == kb1 - 1) mma_commit(accf);
      }
      __syncwarp();
    }
    if (!ok && elect_one()) gemm::drain_mma(drain, abort_flag);
    __syncwarp();
  } else if constexpr (kQuantize) {
    // One task is 256 elements of K of up to four rows: 8 elements of each to a
    // lane, blocks in 4 (MXFP4) or 2 neighbouring lanes.  Tasks run K block
    // after K block; the next one's loads are under way while one is cast.
    constexpr int kLanes = Kind<KIND>::kBlock / 8;
    const int groups = (rows + 3) / 4, tasks = groups * (kb1 - kb0);
    const XT *x = static_cast<const XT *>(p.x) + (int64_t)mt * p.nb * p.ldx;
    const bool g_bad = !(g < __uint_as_float(0x7F800000u));
    const bool odd = lane & 1;
    auto fetch = [&](int t, Pack8<XT> (&v)[4]) {
      const int kbl = t / groups, row0 = (t - kbl * groups) * 4;
      const int64_t k = (int64_t)(kb0 + kbl) * kBK + lane * 8;
      const int in = t < tasks ? (int)max((int64_t)0, min((int64_t)8, p.K - k)) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int valid = row0 + i < rows ? in : 0;
        const XT *at = x + (valid > 0 ? (row0 + i) * p.ldx + k : 0);
        if (p.vec)
          pack8::load<true>(v[i], at, valid);
        else
          v[i].load_some(at, valid);
      }
    };
    Pack8<XT> next[4];
    fetch(warp - 2, next);
    for (int t = warp - 2; t < tasks; t += kQuantWarps) {
      Pack8<XT> y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = next[i];
      fetch(t + kQuantWarps, next);
      const int kbl = t / groups, row0 = (t - kbl * groups) * 4;
      const int s = kbl % p.stages;
      uint32_t m[4], top = 0, byte[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = y[i].amax_bits();
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
        top = max(top, m[i]);
      }
      if (!__any_sync(0xFFFFFFFFu, top >= kCarefulBits || g_bad)) {
        if (KIND == FP4Q_NVFP4) {   // the two lanes of a block find two rows' scales each
          const float t0 = fmaxf(nv_ratio(__uint_as_float(odd ? m[2] : m[0]), g, rg), 0x1p-9f);
          const float t1 = fmaxf(nv_ratio(__uint_as_float(odd ? m[3] : m[1]), g, rg), 0x1p-9f);
          const uint32_t mine =
              (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t0, t1), __NV_SATFINITE, __NV_E4M3);
          const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
          const uint32_t all = odd ? other | mine << 16 : mine | other << 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) byte[i] = (all >> (8 * i)) & 0xFFu;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (row0 + i >= rows) break;
          float d = 0.0f, r;
          if (KIND == FP4Q_MXFP4) {
            byte[i] = mx_byte(m[i]);
            r = mx_reciprocal(byte[i]);
          } else {
            const float2 dr = table.d_r[byte[i]];
            d = dr.x;
            r = dr.y;
          }
          const float2 v[4] = {y[i].pair(0), y[i].pair(1), y[i].pair(2), y[i].pair(3)};
          w[i] = encode8<KIND>(v, d, r);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = encode8_careful<KIND>(y[i].pair(0), y[i].pair(1), y[i].pair(2), y[i].pair(3),
                                       m[i], g, &byte[i]);
      }
      // Not the slot's own barrier: a warp's next task may be several turns of
      // the ring ahead, where a phase's parity does not tell which turn it is.
      if (!wait_counter_all(free_kb, kbl, abort_flag, p.err)) break;
      uint8_t *stage = ring_ptr + s * p.stage_bytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + i;
        if (row >= rows) break;
        // the 128-byte swizzle: 16-byte chunk index xor row of the 8-row group
        *reinterpret_cast<uint32_t *>(stage + kXOff + row * 128 +
                                      ((((lane >> 2) ^ row) & 7) << 4 | (lane & 3) << 2)) = w[i];
        if ((lane & (kLanes - 1)) == 0) {
          const int block = lane / kLanes;   // of this stage
          stage[kSfbOff + (block >> 2) * 512 + row * 16 + (block & 3)] = (uint8_t)byte[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full0 + 8 * s);
    }
  }

  // Partial sums [row of x][row of w] in shared memory (the ring is free: its
  // last MMAs are done), then every rank adds its share of the tile.
  float *part = reinterpret_cast<float *>(ring_ptr);
  if (warp >= 2) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    // in a group some CTAs of a cluster may have no K block: they add zeros
    const bool ok = kb1 > kb0 && wait_bounded_all(accf, 0, abort_flag, p.err);
    tc_fence_after();
    for (int c = 32 * half; c < rows; c += 64) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < rows) part[(c + j) * 128 + quarter * 32 + lane] = ok ? __uint_as_float(r[j]) : 0.0f;
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (p.split > 1) cluster_sync_any();
  {
    float scale = 1.0f;
    if (KIND == FP4Q_NVFP4) scale = __fmul_rn(kQuantize ? g : *p.gx, *p.gw);
    const int total = rows * 32;   // groups of four columns
    const int first = (int)((int64_t)total * rank / p.split);
    const int last = (int)((int64_t)total * (rank + 1) / p.split);
    const uint32_t part_u32 = smem_u32(part);
    const bool whole = p.N % 4 == 0;   // whole groups, 8- or 16-byte aligned (y is)
#pragma unroll 2
    for (int i = first + (int)threadIdx.x; i < last; i += kThreads) {
      const int row = i >> 5, n = (i & 31) * 4;
      float4 t[kMaxSplit];
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < p.split) t[r] = ld_shared_cluster_f4(mapa_shared(part_u32 + 16 * i, r));
      float4 v = t[0];
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r)
        if (r < p.split) v.x += t[r].x, v.y += t[r].y, v.z += t[r].z, v.w += t[r].w;
      if (KIND == FP4Q_NVFP4) {
        v.x = __fmul_rn(v.x, scale), v.y = __fmul_rn(v.y, scale);
        v.z = __fmul_rn(v.z, scale), v.w = __fmul_rn(v.w, scale);
      }
      const int64_t col = (int64_t)nt * 128 + n;
      const int64_t at = ((int64_t)mt * p.nb + row) * p.N + col;
      if (whole) {
        if (col >= p.N) continue;
        if (p.out_bf16)
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + at) =
              make_uint2(pack8::bf16x2(v.x, v.y), pack8::bf16x2(v.z, v.w));
        else
          *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at) = v;
      } else {
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (col + j >= p.N) break;
          if (p.out_bf16)
            static_cast<__nv_bfloat16 *>(p.y)[at + j] = __float2bfloat16_rn(e[j]);
          else
            static_cast<float *>(p.y)[at + j] = e[j];
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync_any();   // no CTA leaves while another may read its sums
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
}

// Shared memory of one CTA, and all of the SM's on-chip memory for two.
template <typename Kernel>
bool set_up(Kernel kernel) {
  return gemm::set_smem(kernel, kSmemBytes) == cudaSuccess &&
         cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared) == cudaSuccess;
}

// Clusters of 1 .. kMaxSplit CTAs that run on the current device with every CTA
// alone on its SM, and that run at once: a cluster keeps to one of the GPU's
// partitions, so fewer CTAs fit as sixes or sevens than singly.  Every
// instantiation has the same block, shared memory and residence, so one kernel
// answers for all.  The query counts one CTA an SM here whatever the shared
// memory; two run, hence twice its answer, and a cluster of seven or eight fits
// on four SMs: as many as fours alone.  Counted, and found by the time's jump as
// tiles are added (1 .. 8): 304, 152, 92, 72, 56, 46, 36, 36 and 304, 152, 97, 74,
// 58, 46, 38, 36.
struct Fit {
  int alone[kMaxSplit], at_once[kMaxSplit];
};

// Null on failure.
const Fit *clusters_at_once() {
  static Fit fits[64];
  static PerDeviceOnce setup;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  const int ok = setup.get([&] {
    Fit &fit = fits[dev];
    auto kernel = split_kernel<FP4Q_MXFP4, void, false>;
    if (!set_up(kernel)) return 0;
    for (int s = 1; s <= kMaxSplit; ++s) {
      Launch q(s, 1, kThreads, kSmemBytes, nullptr, s);
      q.cfg.numAttrs = 2;   // the query wants the cluster size, one included
      if (cudaOccupancyMaxActiveClusters(&fit.alone[s - 1], kernel, &q.cfg) != cudaSuccess ||
          fit.alone[s - 1] < 1)
        return 0;
      fit.at_once[s - 1] = 2 * fit.alone[s - 1];
      if (s >= 7) fit.at_once[s - 1] = std::max(fit.at_once[s - 1], fit.alone[3]);
    }
    return 1;
  });
  return ok == 1 ? &fits[dev] : nullptr;
}

int rows_per_tile(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

// CTAs a tile: the most of which all tiles run at once.  A tile that has to
// wait for a place costs a whole turn: one row, K 8192, 46 tiles as sixes take
// 7.3 us and 47 take 11.9 (as fives 7.5).  Each CTA has a K block at least;
// where CTAs share an SM, four, and eight if a tile has 128 rows, since joining
// the sums of two CTAs an SM costs as much: 16 x 4480 x 2048, 35 tiles, 5.9 us as
// eights and 4.9 as fours, 128 x 4096 x 4096, 32 tiles, 9.9 as eights and 7.9 as
// fours.  Over 890 sizes (M 1-512, N 512-16384, K 1024-16384) the choice is 1.0%
// from the best split on average; farthest where threes are counted low: 16 x
// 12288 x 16384, 96 tiles, 31.8 us as twos and 24.2 as threes.
int split_of(const Fit &fit, int64_t tiles, int64_t k_blocks, int nb) {
  const int64_t least = nb == kMaxRows ? 8 : 4;
  int s = (int)std::min<int64_t>(kMaxSplit, k_blocks);
  while (s > 1 && (fit.at_once[s - 1] < tiles || (fit.alone[s - 1] < tiles && k_blocks < least * s)))
    --s;
  return s;
}

template <int KIND, typename XT, bool GROUPED>
int run_split(const Group<GROUPED> &group, cudaStream_t stream) {
  auto kernel = split_kernel<KIND, XT, GROUPED>;
  static PerDeviceOnce setup;  // per instantiation
  if (setup.get([&] { return set_up(kernel) ? 1 : 0; }) != 1) return FP8Q_ERR_CUDA;
  const int split = group.prob[0].split;
  log_line("  %d products, grid %d in clusters of %d", group.n, group.tile_end[group.n - 1] * split, split);
  return Launch((unsigned)(group.tile_end[group.n - 1] * split), 1, kThreads, kSmemBytes, stream,
                split)
                     .run(kernel, group) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

// Everything of a group but what is only of the quantising launch.
template <bool GROUPED>
int fill_group(Group<GROUPED> &group, int kind, const Product *prod, int n, bool quantized,
               int out_dtype) {
  unsigned int *err = device_error_word();
  const Fit *fit = clusters_at_once();
  if (err == nullptr || fit == nullptr) return FP8Q_ERR_CUDA;
  const int atoms = kind == FP4Q_MXFP4 ? 2 : 4, sf_cols = 8 * atoms;
  group.n = n;
  int64_t tiles = 0, k_blocks = 1;
  int nb = 0;
  for (int i = 0; i < n; ++i) {
    const Product &d = prod[i];
    Args &a = group.prob[i];
    a.M = d.M;
    a.N = d.N;
    a.K = d.K;
    a.gx = d.A.global_scale;
    a.gw = d.B.global_scale;
    a.y = d.C;
    a.nb = rows_per_tile(d.M);
    a.num_k_blocks = (int)((d.K + kBK - 1) / kBK);
    a.num_steps = (int)((d.K + 63) / 64);
    a.atoms_k = (int)num_atoms_k(kind, d.K);
    a.out_bf16 = out_dtype == FP8Q_DT_BF16;
    a.err = err;
    a.m_tiles = (int)((d.M + a.nb - 1) / a.nb);
    a.idesc = idesc_fp4(kind, 128, (uint32_t)a.nb);
    a.stage_bytes = (128 * kBKBytes + 2 * atoms * 512 + 1023) / 1024 * 1024 + a.nb * kBKBytes;
    a.stages = std::min(kMaxStages, (kSmemBytes - kFixedBytes) / a.stage_bytes);
    a.stages = std::min(a.stages, ((int)kTmemCols - std::max(32, a.nb)) / sf_cols);
    tiles += (d.N + 127) / 128 * a.m_tiles;
    if (tiles > INT32_MAX / kMaxSplit) return FP8Q_ERR_INVALID_ARG;
    group.tile_end[i] = (int)tiles;
    k_blocks = std::max<int64_t>(k_blocks, a.num_k_blocks);
    nb = std::max(nb, a.nb);
    Maps &m = group.maps[i];
    if (!make_tmap(&m.w, d.B.data, d.N, d.K, 128) ||
        !make_scale_tmap(&m.sfw, d.B.scales, d.N, a.atoms_k, (uint32_t)atoms))
      return FP8Q_ERR_CUDA;
    if (!quantized) {
      m.x = m.w;   // not used
      m.sfx = m.sfw;
    } else if (!make_tmap(&m.x, d.A.data, d.M, d.K, (uint32_t)a.nb) ||
               !make_scale_tmap(&m.sfx, d.A.scales, d.M, a.atoms_k, (uint32_t)atoms)) {
      return FP8Q_ERR_CUDA;
    }
  }
  const int split = split_of(*fit, tiles, k_blocks, nb);
  for (int i = 0; i < n; ++i) {
    group.prob[i].split = split;
    log_line("launch fp4 split_kernel %lldx%lldx%lld kind %d rows %d tiles %lld split %d stages %d%s%s",
             (long long)prod[i].M, (long long)prod[i].N, (long long)prod[i].K, kind,
             group.prob[i].nb, (long long)tiles, split, group.prob[i].stages,
             quantized ? "" : " quantising x", n > 1 ? " grouped" : "");
  }
  return FP8Q_OK;
}

template <bool GROUPED>
int start_split(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream) {
  Group<GROUPED> group{};
  const int rc = fill_group(group, kind, prod, n, true, out_dtype);
  if (rc != FP8Q_OK) return rc;
  return kind == FP4Q_MXFP4 ? run_split<FP4Q_MXFP4, void>(group, stream)
                            : run_split<FP4Q_NVFP4, void>(group, stream);
}

}  // namespace

double split_cost(int64_t M, int64_t N, int64_t K) {
  const Fit *fit = clusters_at_once();
  if (fit == nullptr) return 0.0;
  const int nb = rows_per_tile(M);
  const int64_t kb = (K + kBK - 1) / kBK;
  const int64_t tiles = (N + 127) / 128 * ((M + nb - 1) / nb);
  const int s = split_of(*fit, tiles, kb, nb);
  const int64_t waves = (tiles + fit->at_once[s - 1] - 1) / fit->at_once[s - 1];
  return (double)waves * (0.45 * (double)((kb + s - 1) / s) + (fit->alone[s - 1] < tiles ? 2.0 : 0.3));
}

int launch_split(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream) {
  return n > 1 ? start_split<true>(kind, prod, n, out_dtype, stream)
               : start_split<false>(kind, prod, n, out_dtype, stream);
}

int launch_split_quantizing(int kind, const void *x, int in_dtype, int64_t ldx,
                            const float *x_amax, const Product &prod, int out_dtype,
                            cudaStream_t stream) {
  Group<false> group{};
  const int rc = fill_group(group, kind, &prod, 1, false, out_dtype);
  if (rc != FP8Q_OK) return rc;
  Args &a = group.prob[0];
  const int64_t size = in_dtype == FP8Q_DT_BF16 ? 2 : 4;
  a.x = x;
  a.ldx = ldx;
  a.x_amax = x_amax;
  a.vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * size % 16 == 0 && prod.K % 8 == 0;
  if (kind == FP4Q_MXFP4)
    return in_dtype == FP8Q_DT_BF16 ? run_split<FP4Q_MXFP4, __nv_bfloat16>(group, stream)
                                    : run_split<FP4Q_MXFP4, float>(group, stream);
  return in_dtype == FP8Q_DT_BF16 ? run_split<FP4Q_NVFP4, __nv_bfloat16>(group, stream)
                                  : run_split<FP4Q_NVFP4, float>(group, stream);
}

}  // namespace fp4
}  // namespace fp8q
