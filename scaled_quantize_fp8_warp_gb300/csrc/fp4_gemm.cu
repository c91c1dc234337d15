// The product of two 4-bit operands, C = A . B^T, on the tensor cores' own
// block scaling (tcgen05.mma kind::mxf4nvf4): every K block's scales are
// copied from shared into tensor memory (tcgen05.cp) ahead of its MMAs, the
// whole K range accumulates in fp32 in tensor memory, and the epilogue
// multiplies by the tensor scales (NVFP4), converts and stores.
//
// CTA pairs (tcgen05.mma.cta_group::2) compute tiles of 256 x 256 or 256 x 384,
// each CTA staging its own 128 rows of A and half of B's rows per 256 elements
// of K (128 bytes a row, 128-byte swizzle).  Each CTA loads the scale atoms of
// its own rows of A and of all rows of B, by tensor maps in which an atom is a
// row of 128 words; the even CTA's copies put both CTAs' into tensor memory.
// Tensor memory: the accumulator, then slots of scales, which leaves no room
// for a second accumulator: the epilogue's warps take it into registers at once
// and release it before they store.
//
// What bounds it: the copies into shared memory, then the MMAs.  8192 cube with
// 256-wide tiles: 183 us NVFP4 and 176 MXFP4, 157 and 144 with the loads taken
// out: 7.6 PFLOP/s, four times the measured bf16 rate, is what MMAs of K = 64
// reach (the dense 4-bit rate the chip is sold at, six times bf16's, has an
// MMA of K = 96, which is not used here).  A fit over sizes gives a 384-wide tile 0.49 us per 256 of K (48 KB a CTA
// for NVFP4, so 15 TB/s over all SMs) and 1.65 us at its end.  Long loops meet
// the board's power limit: 256-wide 398 us at 1.83-1.90 GHz, with operands of
// zeros 369 at 2.07.  In several runs, NVFP4 15872 x 16384 x 4096: 340-344
// us (6.2-6.3 PFLOP/s); 15872 x 4096 x 16384: 295-297 us (7.2); 8192 cube: NVFP4
// 170-193 us, MXFP4 160-173.  15872 x 16384 x 4096 NVFP4 took 654 us with one SM
// a tile, 747 in pairs with instructions issued under a lane comparison, 377
// under elect.sync.  Slower: scales and MMAs in elected blocks of their own (388
// for 376), a wide tile's two column groups handed over in turn (410 for 340),
// one thread for the whole loop (351 for 347).
#include <cuda.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

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

constexpr int kBKBytes = 128;          // bytes of K per stage
constexpr int kBK = 256;               // elements of K per stage

struct Args {
  int64_t M, N;
  int num_m_tiles, num_n_tiles, num_k_blocks;
  int num_steps;            // MMAs of 64 K over all of K
  int atoms_k;              // scale atoms along K
  int group;                // raster: tile rows visited together
  void *C;
  const float *ga, *gb;     // NVFP4 tensor scales
  unsigned int *err;
};

// BN: columns of a tile, 256 or 384.
template <int KIND, int WIDTH, int BN>
struct PairLayout {
  static constexpr int kAtoms = kBK / Kind<KIND>::kAtomK;     // per stage and 128 rows: 2 or 4
  static constexpr int kRowBlocks = BN / 128;                 // of B
  static constexpr int kABytes = 128 * kBKBytes, kBBytes = BN / 2 * kBKBytes;
  static constexpr int kSfaOff = kABytes + kBBytes;
  static constexpr int kSfbOff = kSfaOff + kAtoms * 512;
  static constexpr int kLoadBytes = kSfbOff + kRowBlocks * kAtoms * 512;
  static constexpr int kStageBytes = (kLoadBytes + 1023) / 1024 * 1024;
  // Epilogue warps: 128 (of 256) or 96 (of 384) columns and 32 rows each.
  static constexpr int kEpilogueColumns = BN == 384 ? 96 : 128;
  static constexpr int kEpilogueWarps = 4 * BN / kEpilogueColumns;
  static constexpr int kThreads = 32 * (2 + kEpilogueWarps);
  // rows that allow no vector store pass through shared memory, a 32 x 32
  // block a warp: a stage less
  static constexpr int kTurnBytes = WIDTH == 0 ? kEpilogueWarps * 32 * 33 * 4 : 0;
  static constexpr int kStages =
      (BN == 384 ? 4 : (KIND == FP4Q_MXFP4 ? 6 : 5)) - (WIDTH == 0 ? 1 : 0);
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kBarBytes = 8 * (2 * kStages + 3);
  static constexpr int kSmemBytes = kRingBytes + kTurnBytes + kBarBytes + 16 + 1024;
  // Tensor memory: the accumulator, then slots of scales, one per stage where
  // that fits (NVFP4 at 384 columns: two).
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSfCols = 4 * kAtoms * (1 + kRowBlocks);
  static constexpr int kSlots =
      (int)((kTmemCols - BN) / kSfCols) < kStages ? (int)((kTmemCols - BN) / kSfCols) : kStages;
  static_assert(kSlots >= 2, "a block's scales arrive while another's are read");
  static_assert(kSmemBytes <= 227 * 1024, "the ring fits in shared memory");
};

// One K block in the ring slot at `sa` (A, B, A's atoms, B's atoms row block
// after row block), by one elected thread: scales into tensor memory at sf,
// then up to four steps of 64 K.  A step is one MMA of N = 256 and, for tiles
// 384 wide, one of N = 128.  The last block may hold fewer steps: K past the
// matrix would multiply zeros with scales that were not loaded.
template <int KIND, int BN>
__device__ __forceinline__ void issue_block(uint32_t sa, uint32_t d_tmem, uint32_t sf, int steps,
                                            bool first) {
  using L = PairLayout<KIND, 32, BN>;   // offsets do not depend on the width of stores
  constexpr int kAtoms = L::kAtoms, kRowBlocks = BN / 128;
  const uint32_t sfa = sf, sfb = sf + 4 * kAtoms;
  const uint64_t atom = sdesc_plain(sa + L::kSfaOff, 128);   // + 32 per atom (512 bytes >> 4)
#pragma unroll
  for (int a = 0; a < kAtoms; ++a) {
    tmem_cp_32x128b_x4_pair(sfa + 4 * a, atom + 32 * a);
#pragma unroll
    for (int h = 0; h < kRowBlocks; ++h)
      tmem_cp_32x128b_x4_pair(sfb + 4 * (kRowBlocks * a + h), atom + 32 * (kAtoms * (1 + h) + a));
  }
  constexpr uint32_t idesc = idesc_fp4(KIND, 256, 256), idesc128 = idesc_fp4(KIND, 256, 128);
  const uint64_t ad = sdesc_k(sa, gemm::kSwzSBO, gemm::kSwzMode);
  const uint64_t bd = sdesc_k(sa + L::kABytes, gemm::kSwzSBO, gemm::kSwzMode);
  const auto step = [&](int k) {
    const int a = KIND == FP4Q_MXFP4 ? k >> 1 : k;
    const uint32_t half = KIND == FP4Q_MXFP4 ? 2u * (k & 1) : 0u;   // of the scale word
    const uint32_t pick = (half << 29) | (half << 4), acc = (!first || k > 0) ? 1u : 0u;
    mma_fp4_pair<KIND>(d_tmem, ad + 2 * k, bd + 2 * k, idesc | pick, sfa + 4 * a,
                       sfb + 4 * kRowBlocks * a, acc);
    if (BN == 384)   // B's rows 128-191 of each CTA
      mma_fp4_pair<KIND>(d_tmem + 256, ad + 2 * k, bd + 2 * k + (128 * kBKBytes >> 4),
                         idesc128 | pick, sfa + 4 * a, sfb + 4 * (kRowBlocks * a + 2), acc);
  };
  if (steps >= 4) {   // without a test per step: those alone cost NVFP4 7%
#pragma unroll
    for (int k = 0; k < 4; ++k) step(k);
  } else {
    for (int k = 0; k < steps; ++k) step(k);
  }
}

// 32 consecutive results of row m from column n0, as the words they are stored
// as.  WIDTH: every row of C starts on a boundary of so many bytes (32 or 16),
// and whole groups of that size are stored at once.
template <typename T, int WIDTH>
__device__ __forceinline__ void store32(T *C, int64_t N, int64_t m, int64_t n0,
                                        const uint32_t (&r)[8 * sizeof(T)]) {
  T *row = C + m * N + n0;
  constexpr int kWords = WIDTH / 4, kGroup = WIDTH / (int)sizeof(T);
#pragma unroll
  for (int g = 0; g < 32 / kGroup; ++g) {
    if (n0 + g * kGroup >= N) break;
    uint32_t w[kWords];
#pragma unroll
    for (int h = 0; h < kWords; ++h) w[h] = r[g * kWords + h];
    if constexpr (WIDTH == 32)
      store_32b(row + g * kGroup, w);
    else
      __stcs(reinterpret_cast<uint4 *>(row + g * kGroup), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// The same for a warp's 32 rows from m0 where rows start anywhere: turned in
// shared memory so that lanes store neighbouring elements (stores of single
// elements by the lanes that own the rows measured 33 us more on 2048 x 650).
template <typename T>
__device__ __forceinline__ void store32_turned(T *C, int64_t M, int64_t N, int64_t m0, int64_t n0,
                                               const uint32_t (&r)[8 * sizeof(T)], uint32_t *turn) {
  constexpr int kWords = 8 * (int)sizeof(T);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kWords; ++j) turn[lane * (kWords + 1) + j] = r[j];
  __syncwarp();
  T *at = C + m0 * N + n0 + lane;
  const T *from = reinterpret_cast<const T *>(turn) + lane;
  const int rows = (int)min((int64_t)32, M - m0);
  if (n0 + lane < N)
    for (int i = 0; i < rows; ++i) at[i * N] = from[i * (kWords + 1) * (4 / (int)sizeof(T))];
  __syncwarp();
}

struct PairMaps {
  CUtensorMap a, b, b64, sfa, sfb;   // b64: boxes of 64 rows of B, for tiles 384 wide
};

// The products of one launch, their tiles numbered one product after the other,
// so that only the last wave of all is partial.  A launch of one (GROUPED
// false) reads it at constant offsets.
template <bool GROUPED>
struct PairGroup {
  static constexpr int kMax = GROUPED ? kGroupMax : 1;
  int n;
  int unit_end[kMax];
  Args prob[kMax];
  PairMaps maps[kMax];
};

template <bool GROUPED>
__device__ __forceinline__ int group_coords(const PairGroup<GROUPED> &g, int u, int &mu, int &nt) {
  int q = 0;
  if (GROUPED) {
    while (q + 1 < g.n && u >= g.unit_end[q]) ++q;
    if (q > 0) u -= g.unit_end[q - 1];
  }
  const Args &p = g.prob[q];
  gemm::tile_coords(u, (p.num_m_tiles + 1) / 2, p.num_n_tiles, mu, nt, p.group, 0);
  return q;
}

template <int KIND, typename T, int WIDTH, int BN, bool GROUPED>
__global__ void __launch_bounds__(PairLayout<KIND, WIDTH, BN>::kThreads, 1)
    gemm_pair_kernel(const __grid_constant__ PairGroup<GROUPED> grp) {
  using L = PairLayout<KIND, WIDTH, BN>;
  constexpr int kStages = L::kStages;
  constexpr uint16_t kBoth = 3;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + L::kRingBytes + L::kTurnBytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
  const uint32_t accf = bars + 8 * (2 * kStages), acce = accf + 8, drain = acce + 8;
  const uint32_t slot = bars + L::kBarBytes;
  uint8_t *slot_ptr = smem_raw + (slot - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: issues the pair's MMAs
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
    mbar_init(acce, 2 * L::kEpilogueWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    for (int q = 0; q < (GROUPED ? grp.n : 1); ++q) {
      prefetch_tmap(&grp.maps[q].a);
      prefetch_tmap(&grp.maps[q].b);
      if (BN == 384) prefetch_tmap(&grp.maps[q].b64);
      prefetch_tmap(&grp.maps[q].sfa);
      prefetch_tmap(&grp.maps[q].sfb);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(slot, L::kTmemCols);
    tmem_relinquish_pair();
  }
  follow_previous();
  allow_next();
  tc_fence_before();
  __syncthreads();
  cluster_sync_any();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);
  // One allocation serves the pair: both CTAs must hold the same address.
  // Otherwise neither does any work (a symmetric decision, no waiting).
  const bool paired = ld_shared_cluster_u32(mapa_shared(slot, rank ^ 1u)) == tmem_base;
  unsigned int *const err = grp.prob[0].err;
  if (!paired && threadIdx.x == 0) atomicOr(err, 4u);

  const int total = grp.unit_end[GROUPED ? grp.n - 1 : 0];
  const int unit0 = blockIdx.x / 2, unit_step = gridDim.x / 2;

  if (!paired) {
  } else if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = unit0; u < total && ok; u += unit_step) {
        int mu, nt;
        const int q = group_coords(grp, u, mu, nt);
        const PairMaps &maps = grp.maps[q];
        const int num_k_blocks = grp.prob[q].num_k_blocks, atoms_k = grp.prob[q].atoms_k;
        // past the last M tile (odd count): re-read that tile's A, store nothing
        const int mt = min(2 * mu + (int)rank, grp.prob[q].num_m_tiles - 1);
        for (int kb = 0; kb < num_k_blocks; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + s * L::kStageBytes;
          const uint32_t full_even = mapa_shared(full0 + 8 * s, 0);
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * L::kLoadBytes);
          tma_load_2d_pair(sa, &maps.a, kb * kBKBytes, mt * 128, full_even);
          tma_load_2d_pair(sa + L::kABytes, &maps.b, kb * kBKBytes, nt * BN + (int)rank * 128,
                           full_even);
          if (BN == 384)
            tma_load_2d_pair(sa + L::kABytes + 128 * kBKBytes, &maps.b64, kb * kBKBytes,
                             nt * BN + 256 + (int)rank * 64, full_even);
          // Atoms past the last of a row block are the next block's or zeros;
          // no MMA step reads them.
          const int ka = kb * L::kAtoms;
          tma_load_2d_pair(sa + L::kSfaOff, &maps.sfa, 0, mt * atoms_k + ka, full_even);
#pragma unroll
          for (int h = 0; h < L::kRowBlocks; ++h)
            tma_load_2d_pair(sa + L::kSfbOff + h * L::kAtoms * 512, &maps.sfb, 0,
                             (L::kRowBlocks * nt + h) * atoms_k + ka, full_even);
        }
      }
      // every slot's last release (the even CTA's commits) has arrived here
      for (uint32_t j = 0, jt = it; ok && j < (uint32_t)kStages; ++j, ++jt)
        ok = wait_bounded(empty0 + 8 * (jt % kStages), ((jt / kStages) & 1u) ^ 1u, abort_flag,
                          err);
      if (!ok) {
        // aborting: give copies already issued (their barrier may be the
        // other CTA's) a millisecond to land before the CTA can leave
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    uint32_t it = 0, acc_it = 0;
    bool ok = true;
    for (int u = unit0; u < total && ok; u += unit_step, ++acc_it) {
      int mu, nt;
      const int q = group_coords(grp, u, mu, nt);
      const int num_k_blocks = grp.prob[q].num_k_blocks, num_steps = grp.prob[q].num_steps;
      if (!wait_bounded_all(acce, (acc_it & 1u) ^ 1u, abort_flag, err)) break;
      tc_fence_after();
      for (int kb = 0; kb < num_k_blocks; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        if (!wait_bounded_all(full0 + 8 * s, ph, abort_flag, err)) {
          ok = false;
          break;
        }
        // the MMAs that read this slot of scales last are done
        if (L::kSlots < kStages && it >= (uint32_t)L::kSlots) {
          const uint32_t old = it - L::kSlots;
          if (!wait_bounded_all(empty0 + 8 * (old % kStages), (old / kStages) & 1u, abort_flag,
                                err)) {
            ok = false;
            break;
          }
        }
        tc_fence_after();
        if (elect_one()) {
          issue_block<KIND, BN>(ring + s * L::kStageBytes, tmem_base,
                                tmem_base + BN + L::kSfCols * (it % L::kSlots),
                                num_steps - 4 * kb, kb == 0);
          mma_commit_pair_multicast(empty0 + 8 * s, kBoth);
          if (kb == num_k_blocks - 1) mma_commit_pair_multicast(accf, kBoth);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      mma_commit_pair(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 200000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
  } else {
    // Warp w drains TMEM lane quarter w % 4, columns [W h, W h + W) with W =
    // kEpilogueColumns and h = (w - 2) / 4, of this CTA's 128 rows.
    constexpr int kChunks = L::kEpilogueColumns / 32;
    const int quarter = warp & 3, first = (warp - 2) / 4 * L::kEpilogueColumns;
    const uint32_t acce_even = mapa_shared(acce, 0);
    uint32_t acc_it = 0;
    for (int u = unit0; u < total; u += unit_step, ++acc_it) {
      int mu, nt;
      const int q = group_coords(grp, u, mu, nt);
      const int64_t M = grp.prob[q].M, N = grp.prob[q].N;
      T *const C = static_cast<T *>(grp.prob[q].C);
      const float g = KIND == FP4Q_NVFP4 ? __fmul_rn(*grp.prob[q].ga, *grp.prob[q].gb) : 1.0f;
      if (!wait_bounded_warp(accf, acc_it & 1u, abort_flag, err)) break;
      tc_fence_after();
      // bf16 results are rounded as they come, two to a register: fewer live
      constexpr int kRegs = sizeof(T) == 2 ? 16 : 32;
      uint32_t r[kChunks][kRegs];
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t t[2][32];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (c + k < kChunks)
            tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + first + (c + k) * 32, t[k]);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (c + k < kChunks)
#pragma unroll
            for (int j = 0; j < kRegs; ++j) {
              if constexpr (sizeof(T) == 2) {
                float a = __uint_as_float(t[k][2 * j]), b = __uint_as_float(t[k][2 * j + 1]);
                if (KIND == FP4Q_NVFP4) a = __fmul_rn(a, g), b = __fmul_rn(b, g);
                r[c + k][j] = pack8::bf16x2(a, b);
              } else {
                float a = __uint_as_float(t[k][j]);
                if (KIND == FP4Q_NVFP4) a = __fmul_rn(a, g);
                r[c + k][j] = __float_as_uint(a);
              }
            }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {   // the accumulator is free for the next tile
        if (rank == 0)
          mbar_arrive(acce);
        else
          mbar_arrive_cluster(acce_even);
      }
      const int64_t m0 = (int64_t)(2 * mu + (int)rank) * 128 + quarter * 32;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int64_t n0 = (int64_t)nt * BN + first + c * 32;
        if (n0 >= N || m0 >= M) break;
        if constexpr (WIDTH == 0)
          store32_turned(C, M, N, m0, n0, r[c],
                         reinterpret_cast<uint32_t *>(smem_raw + (ring - raw) + L::kRingBytes) +
                             (warp - 2) * 32 * 33);
        else if (m0 + lane < M)
          store32<T, WIDTH>(C, N, m0 + lane, n0, r[c]);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_any();  // neither CTA leaves while the other may still signal it
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem_base, L::kTmemCols);
}

template <int KIND, typename T, int WIDTH, int BN, bool GROUPED>
int run_pair(const PairGroup<GROUPED> &grp, cudaStream_t stream) {
  using L = PairLayout<KIND, WIDTH, BN>;
  auto kernel = gemm_pair_kernel<KIND, T, WIDTH, BN, GROUPED>;
  static PerDeviceOnce setup;  // per instantiation: the pairs that fit at once, 0 on failure
  const int pairs = setup.get([&] {
    if (gemm::set_smem(kernel, L::kSmemBytes) != cudaSuccess) return 0;
    Launch q(2 * (sm_count() / 2), 1, L::kThreads, L::kSmemBytes, stream, 2);
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q.cfg) == cudaSuccess ? n : 0;
  });
  if (pairs < 1) return FP8Q_ERR_CUDA;
  const int units = grp.unit_end[grp.n - 1];
  log_line("  %d products, %d tiles, grid %d in pairs", grp.n, units, 2 * std::min(units, pairs));
  return Launch(2 * std::min(units, pairs), 1, L::kThreads, L::kSmemBytes, stream, 2)
                     .run(kernel, grp) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

// Bytes that every row of C starts on: 32, 16 or 0 (neither).
int row_width(const void *C, int64_t N, int64_t size) {
  if (N * size % 32 == 0 && reinterpret_cast<uintptr_t>(C) % 32 == 0) return 32;
  return N * size % 16 == 0 ? 16 : 0;
}

template <int KIND, int BN, bool GROUPED>
int fill_group(PairGroup<GROUPED> &grp, const Product *prod, int n) {
  constexpr int kAtoms = PairLayout<KIND, 32, BN>::kAtoms;
  unsigned int *err = device_error_word();
  if (err == nullptr) return FP8Q_ERR_CUDA;
  grp.n = n;
  int64_t units = 0;
  for (int i = 0; i < n; ++i) {
    const Product &d = prod[i];
    Args &a = grp.prob[i];
    a.M = d.M;
    a.N = d.N;
    a.num_m_tiles = (int)((d.M + 127) / 128);
    a.num_n_tiles = (int)((d.N + BN - 1) / BN);
    a.num_k_blocks = (int)((d.K + kBK - 1) / kBK);
    a.num_steps = (int)((d.K + 63) / 64);
    a.atoms_k = (int)num_atoms_k(KIND, d.K);
    a.group = 8;
    a.C = d.C;
    a.ga = d.A.global_scale;
    a.gb = d.B.global_scale;
    a.err = err;
    units += (int64_t)((a.num_m_tiles + 1) / 2) * a.num_n_tiles;
    if (units > INT32_MAX / 2) return FP8Q_ERR_INVALID_ARG;
    grp.unit_end[i] = (int)units;
    PairMaps &m = grp.maps[i];
    if (!make_tmap(&m.a, d.A.data, d.M, d.K, 128) || !make_tmap(&m.b, d.B.data, d.N, d.K, 128) ||
        !make_scale_tmap(&m.sfa, d.A.scales, d.M, a.atoms_k, kAtoms) ||
        !make_scale_tmap(&m.sfb, d.B.scales, d.N, a.atoms_k, kAtoms) ||
        (BN == 384 && !make_tmap(&m.b64, d.B.data, d.N, d.K, 64)))
      return FP8Q_ERR_CUDA;
  }
  return FP8Q_OK;
}

template <int KIND, typename T, int WIDTH, int BN, bool GROUPED>
int start_pair(const Product *prod, int n, cudaStream_t stream) {
  PairGroup<GROUPED> grp{};
  const int rc = fill_group<KIND, BN>(grp, prod, n);
  return rc == FP8Q_OK ? run_pair<KIND, T, WIDTH, BN>(grp, stream) : rc;
}

template <int KIND, typename T, bool GROUPED>
int launch_pair(const Product *prod, int n, int width, bool wide, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (wide) return start_pair<KIND, T, 32, 384, GROUPED>(prod, n, stream);
  }
  if (width == 32) return start_pair<KIND, T, 32, 256, GROUPED>(prod, n, stream);
  if (width == 16) return start_pair<KIND, T, 16, 256, GROUPED>(prod, n, stream);
  return start_pair<KIND, T, 0, 256, GROUPED>(prod, n, stream);
}

// The products of a launch on CTA pairs.
int launch_pairs(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream) {
  const bool bf16 = out_dtype == FP8Q_DT_BF16;
  // Tiles 384 wide where they take less, by a model fitted to both widths on a
  // busy device: a wave (of as many tiles as there are pairs) takes 0.487 us
  // per 256 of K and 1.65 us at 384, 0.354 and 1.38 at 256.  Only for bf16 rows
  // on 32 bytes: the others' stores need more registers than 576 threads have
  // (8192 x 8200 x 4096 bf16: 110 us at 256, 121 at 384; fp32 402 against 460
  // us at 15872 x 16384 x 4096).
  int width = 32;
  const int64_t pairs = sm_count() / 2;
  double cost[2] = {0.0, 0.0}, waves[2] = {0.0, 0.0};
  for (int i = 0; i < n; ++i) {
    width = std::min(width, row_width(prod[i].C, prod[i].N, bf16 ? 2 : 4));
    const double kb = (double)((prod[i].K + kBK - 1) / kBK);
    for (int w = 0; w < 2; ++w) {
      const int64_t bn = w ? 384 : 256;
      const double tiles = (double)((prod[i].M + 255) / 256 * ((prod[i].N + bn - 1) / bn));
      waves[w] += tiles / (double)pairs;
      cost[w] += tiles / (double)pairs * (w ? 0.487 * kb + 1.65 : 0.354 * kb + 1.38);
    }
  }
  // the last wave is a whole one
  for (int w = 0; w < 2; ++w) cost[w] *= std::ceil(waves[w]) / waves[w];
  const bool wide = bf16 && width == 32 && cost[1] < cost[0];
  for (int i = 0; i < n; ++i)
    log_line("launch fp4 gemm_pair_kernel %lldx%lldx%lld kind %d tile 256x%d out %d%s", (long long)prod[i].M,
             (long long)prod[i].N, (long long)prod[i].K, kind, wide ? 384 : 256, out_dtype,
             n > 1 ? " grouped" : "");
  if (kind == FP4Q_MXFP4) {
    if (n > 1)
      return bf16 ? launch_pair<FP4Q_MXFP4, __nv_bfloat16, true>(prod, n, width, wide, stream)
                  : launch_pair<FP4Q_MXFP4, float, true>(prod, n, width, wide, stream);
    return bf16 ? launch_pair<FP4Q_MXFP4, __nv_bfloat16, false>(prod, n, width, wide, stream)
                : launch_pair<FP4Q_MXFP4, float, false>(prod, n, width, wide, stream);
  }
  if (n > 1)
    return bf16 ? launch_pair<FP4Q_NVFP4, __nv_bfloat16, true>(prod, n, width, wide, stream)
                : launch_pair<FP4Q_NVFP4, float, true>(prod, n, width, wide, stream);
  return bf16 ? launch_pair<FP4Q_NVFP4, __nv_bfloat16, false>(prod, n, width, wide, stream)
              : launch_pair<FP4Q_NVFP4, float, false>(prod, n, width, wide, stream);
}

// Which kernel a product runs on: how many microseconds the split kernel is
// expected to save over CTA pairs.  Up to 64 rows reading B once is the work,
// and the split kernel does little else.  Past that, by a model fitted to both
// kernels timed alone on some 180 shapes (M 128-2048, N 256-12288, K
// 512-16384): beyond a common 6.5 us a wave of 256 x 256 tiles takes 0.33 us
// per 256 of K; a wave of split tiles 0.45 us per 256 of each CTA's K, and 2 us
// (0.3 us where every CTA has an SM to itself) to join the sums.  Both sides of
// the line: 256 x 4096 x 16384 pairs 27.7 us, split 16.6; 512 x 12288 x 4096 pairs
// 18.5 us, split 25.9.  Over 670 sizes (M 65-1024, N 520-12288, K 1024-16384)
// with x cast just before, the choice of kernel and split is 1.8% from the best
// on average; at worst 27% (512 x 520 x 2010, 13.1 us for 10.3).
double split_saves(const Product &d) {
  if (d.M <= 64) return 1e9;
  const int64_t pairs = sm_count() / 2;
  const int64_t waves = ((d.M + 255) / 256 * ((d.N + 255) / 256) + pairs - 1) / pairs;
  return 0.33 * (double)waves * (double)((d.K + kBK - 1) / kBK) - split_cost(d.M, d.N, d.K);
}

// What one launch more costs: where those of a call's products that pairs suit
// better lose less than this together, they join the others' split launch (333
// x 650 x 1031, all three of a training step: 13.1 us the third alone after 10.3
// us the other two, 12 us in one).
constexpr double kLaunchCost = 3.0;

}  // namespace

bool make_tmap(CUtensorMap *m, const void *base, int64_t rows, int64_t K, uint32_t box_rows) {
  const uint64_t bytes = (uint64_t)row_bytes(K);
  return make_tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, bytes, (uint64_t)rows, bytes,
                      kBKBytes, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_scale_tmap(CUtensorMap *m, const uint8_t *scales, int64_t rows, int64_t atoms_k,
                     uint32_t box) {
  return make_tmap_2d(m, scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128,
                      (uint64_t)((rows + 127) / 128 * atoms_k), 512, 128, box,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool product_fits(int kind, int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0) return true;   // no kernel runs
  const int64_t longest = std::max(M, N);
  // a launch of three products numbers the tiles of all, and CTAs of up to eight a tile
  return longest <= INT32_MAX - 1024 && K <= INT32_MAX - 1024 &&
         (M + 255) / 128 * ((N + 511) / 128) <= INT32_MAX / 32 &&
         (longest + 511) / 128 * (num_atoms_k(kind, K) + 4) <= INT32_MAX;
}

int launch_products(int kind, const Product *prod, int n, int out_dtype, cudaStream_t stream) {
  Product todo[kGroupMax];
  double saves[kGroupMax], loss = 0.0;   // of those that pairs suit better
  int count = 0;
  for (int i = 0; i < n; ++i) {
    const Product &d = prod[i];
    if (d.M == 0 || d.N == 0) continue;
    if (d.K == 0) {
      if (cudaMemsetAsync(d.C, 0, (size_t)(d.M * d.N) * (out_dtype == FP8Q_DT_BF16 ? 2 : 4), stream) !=
          cudaSuccess)
        return FP8Q_ERR_CUDA;
      continue;
    }
    todo[count] = d;
    saves[count] = split_saves(d);
    if (saves[count] <= 0.0) loss -= saves[count];
    ++count;
  }
  // those of the split kernel first
  int split = 0;
  for (int i = 0; i < count; ++i)
    if (saves[i] > 0.0) {
      std::swap(todo[split], todo[i]);
      ++split;
    }
  if (split > 0 && loss < kLaunchCost) split = count;
  if (split > 0) {
    const int rc = launch_split(kind, todo, split, out_dtype, stream);
    if (rc != FP8Q_OK) return rc;
  }
  return count > split ? launch_pairs(kind, todo + split, count - split, out_dtype, stream) : FP8Q_OK;
}

}  // namespace fp4
}  // namespace fp8q
