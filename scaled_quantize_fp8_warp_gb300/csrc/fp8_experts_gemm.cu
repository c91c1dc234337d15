// The products of a layer of experts in MXFP8, C_e = B_e . A_e^T for every
// group e, on the tensor cores' own block scaling (tcgen05.mma
// kind::mxf8f6f4): scales go from shared into tensor memory ahead of each K
// block's MMAs, the whole contraction accumulates in fp32 in tensor memory.
//
// The side whose row count is known on the host (a weight's output rows, or
// x's columns for the weights' gradient) is the MMA's M: 256 rows a tile, 128
// in each CTA of a pair (cta_group::2).  The side whose count the router
// decided is its N, up to 256 rows a tile and as few as 32: a group of a few
// rows costs MMAs and loads of 32 rows and not of 256.  The result comes out
// with a column of C in every lane, so a warp stores 32 neighbouring columns.
//
// Persistent: each CTA finds from the offsets where every group's tiles start
// in the numbering of all tiles, and works on every grid-th one.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp4_ptx.cuh"
#include "fp8_experts.h"
#include "fp8_pack8.cuh"
#include "fp8q_gemm_common.cuh"

namespace fp8q {
namespace experts {
namespace {

using namespace ptx;

constexpr int kBK = 128;          // bytes = elements of K per stage
constexpr int kMaxN = 256;        // rows of B per tile
constexpr int kBoxRows = 16;      // rows of B per load of a tile that is not full
constexpr int kRaster = 8;        // tiles of B visited together
constexpr int kMostTiles = INT32_MAX / 2;   // of a launch

struct PairMaps {
  CUtensorMap a, b, b16, sfa, sfb;   // b16: boxes of 16 rows
};

struct Layout {
  static constexpr int kABytes = 128 * kBK, kBBytes = kMaxN / 2 * kBK;
  static constexpr int kSfaOff = kABytes + kBBytes, kSfbOff = kSfaOff + 512;
  static constexpr int kStageBytes = (kSfbOff + 2 * 512 + 1023) / 1024 * 1024;
  static constexpr int kStages = 6;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kBarBytes = 8 * (2 * kStages + 3);
  static constexpr int kTileBytes = (FP8Q_EXPERTS_MAX + 1) * 4;   // first tile of every group
  static constexpr int kSmemBytes = kRingBytes + kBarBytes + 16 + kTileBytes + 1024;
  static constexpr uint32_t kTmemCols = 512, kSfCols = 16;
  static_assert(kSmemBytes <= 227 * 1024, "the ring fits in shared memory");
  static_assert(kMaxN + kSfCols * kStages <= kTmemCols, "scale slots fit in tensor memory");
};
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 32 * (2 + kEpilogueWarps);

// One tile: what of A, B and K it takes, and where its result goes.
struct Tile {
  int a_row, b_row;        // first rows of A and of B
  int k_block, num_k;      // K blocks
  int64_t a_atom, b_atom;  // scale atom of the first rows and the first K block
  int n, valid;            // rows of B: as the MMA takes them (a multiple of 32), and those that count
  int col;                 // first column of C
  int64_t c_row;           // first row of C
};

// Tiles of a group of so many rows.
__device__ __forceinline__ long long tiles_of(const ProductArgs &p, int rows) {
  const int b = p.by_rows ? rows : p.b_rows;
  return (long long)((b + kMaxN - 1) / kMaxN) * ((p.a_rows + 255) / 256);
}

__device__ __forceinline__ Tile find_tile(const ProductArgs &p, const int *first, int u) {
  int lo = 0, hi = p.groups.count;   // first[lo] <= u < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  const int e = lo;
  const int2 group = group_rows(p.groups, e);
  const int block = first_block(p.groups, e, group.x);
  const int rows = p.by_rows ? group.y : p.b_rows;
  int bt, at;
  gemm::tile_coords(u - first[e], (rows + kMaxN - 1) / kMaxN, (p.a_rows + 255) / 256, bt, at,
                    kRaster, 0);
  Tile t;
  t.col = at * 256;
  t.valid = min(kMaxN, rows - bt * kMaxN);
  t.n = (t.valid + 31) / 32 * 32;
  if (p.by_rows) {
    t.a_row = p.a_row * e + t.col;
    t.b_row = group.x + bt * kMaxN;
    t.k_block = p.a_k * e;
    t.num_k = (p.k + kBK - 1) / kBK;
    t.a_atom = (int64_t)(p.a_block * e + 2 * at) * p.a.atoms_k + t.k_block;
    t.b_atom = (int64_t)(block + 2 * bt) * p.b.atoms_k;
    t.c_row = group.x + bt * kMaxN;
  } else {
    t.a_row = t.col;
    t.b_row = bt * kMaxN;
    t.k_block = block;
    t.num_k = (group.y + kBK - 1) / kBK;
    t.a_atom = (int64_t)(2 * at) * p.a.atoms_k + block;
    t.b_atom = (int64_t)(2 * bt) * p.b.atoms_k + block;
    t.c_row = (int64_t)e * p.b_rows + bt * kMaxN;
  }
  return t;
}

// One K block in the ring slot at `sa`, by one elected thread: scales into
// tensor memory at sf, then four MMAs of K = 32.
__device__ __forceinline__ void issue_block(uint32_t sa, uint32_t d_tmem, uint32_t sf,
                                            uint32_t idesc, bool second, bool first) {
  const uint64_t atom = sdesc_plain(sa + Layout::kSfaOff, 128);   // + 32 per atom
  tmem_cp_32x128b_x4_pair(sf, atom);
  tmem_cp_32x128b_x4_pair(sf + 4, atom + 32);
  if (second) tmem_cp_32x128b_x4_pair(sf + 8, atom + 64);
  const uint64_t ad = sdesc_k(sa, gemm::kSwzSBO, gemm::kSwzMode);
  const uint64_t bd = sdesc_k(sa + Layout::kABytes, gemm::kSwzSBO, gemm::kSwzMode);
#pragma unroll
  for (int k = 0; k < 4; ++k)   // step k uses byte k of each scale word
    mma_mxf8f6f4_pair(d_tmem, ad + 2 * k, bd + 2 * k, idesc | ((uint32_t)k << 29) | ((uint32_t)k << 4),
                      sf, sf + 4, (!first || k > 0) ? 1u : 0u);
}

// 32 rows of B in one column of C, as they are kept for storing: bf16 results
// two rows to a register.
template <typename T>
struct Column {
  static constexpr int kRegs = 8 * sizeof(T);
  uint32_t r[kRegs];
  __device__ __forceinline__ void take(const uint32_t (&v)[32]) {
#pragma unroll
    for (int j = 0; j < kRegs; ++j)
      r[j] = sizeof(T) == 4 ? v[j]
                            : pack8::bf16x2(__uint_as_float(v[2 * j % 32]), __uint_as_float(v[(2 * j + 1) % 32]));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < kRegs; ++j) r[j] = 0u;
  }
  // Column m of C from row c_row on, `count` rows of it; lanes hold
  // neighbouring columns.
  __device__ __forceinline__ void store(T *C, int64_t ld, int64_t c_row, int m, int columns,
                                        int count) const {
    if constexpr (sizeof(T) == 4) {
      if (m >= columns) return;
      float *at = reinterpret_cast<float *>(C) + c_row * ld + m;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < count) __stcs(at + j * ld, __uint_as_float(r[j]));
    } else {
      // neighbouring lanes swap halves: the even one stores both their columns
      // of an even row, the odd one those of the row after it (columns % 16 == 0)
      const bool odd = threadIdx.x & 1;
      uint32_t *at = reinterpret_cast<uint32_t *>(C + (c_row + odd) * ld + (m & ~1));
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, r[j], 1);
        const uint32_t w = __byte_perm(r[j], other, odd ? 0x3276 : 0x5410);
        if (2 * j + odd < count && m < columns) __stcs(at + j * ld, w);
      }
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ ProductArgs p,
                   unsigned int *err) {
  using L = Layout;
  constexpr int kStages = L::kStages;
  constexpr uint16_t kBoth = 3;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + L::kRingBytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
  const uint32_t accf = bars + 8 * (2 * kStages), acce = accf + 8, drain = acce + 8;
  const uint32_t slot = bars + L::kBarBytes;
  uint8_t *slot_ptr = smem_raw + (slot - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);
  int *first = reinterpret_cast<int *>(slot_ptr + 16);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: issues the pair's MMAs
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
    mbar_init(acce, 2 * kEpilogueWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.b16);
    prefetch_tmap(&maps.sfa);
    prefetch_tmap(&maps.sfb);
  }
  if (warp == 1) {
    tmem_alloc_pair(slot, L::kTmemCols);
    tmem_relinquish_pair();
  }
  follow_previous();
  allow_next();
  if (warp == 2) {   // where every group's tiles start: a lane has a run of groups
    const int E = p.groups.count, per = (E + 31) / 32;
    const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
    long long sum = 0;
    for (int e = e0; e < e1; ++e) sum += tiles_of(p, group_rows(p.groups, e).y);
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long other = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += other;
    }
    // more than the host allows for come from offsets that are no offsets: nothing is done
    const bool fits = __shfl_sync(0xFFFFFFFFu, upto, 31) <= kMostTiles;
    long long at = fits ? upto - sum : 0;
    for (int e = e0; e < e1; ++e) {
      first[e] = (int)at;
      if (fits) at += tiles_of(p, group_rows(p.groups, e).y);
    }
    if (lane == 31) first[E] = fits ? (int)upto : 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_any();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);
  // One allocation serves the pair: both CTAs must hold the same address.
  // Otherwise neither does any work (a symmetric decision, no waiting).
  const bool paired = ld_shared_cluster_u32(mapa_shared(slot, rank ^ 1u)) == tmem_base;
  if (!paired && threadIdx.x == 0) atomicOr(err, 4u);

  const int total = first[p.groups.count];
  const int unit0 = blockIdx.x / 2, unit_step = gridDim.x / 2;

  if (!paired) {
  } else if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      const int a_blocks = (p.a_rows + 127) / 128;   // 128-row blocks of a group's A
      for (int u = unit0; u < total && ok; u += unit_step) {
        const Tile t = find_tile(p, first, u);
        // past the last block of A (odd count): the even CTA's scales again, nothing is stored
        const int64_t sfa = t.a_atom + (t.col / 128 + (int)rank < a_blocks ? (int)rank : 0) * (int64_t)p.a.atoms_k;
        const int half = t.n / 2, second = t.n > 128;
        const uint32_t bytes = L::kABytes + (uint32_t)half * kBK + 512u * (2u + second);
        for (int kb = 0; kb < t.num_k; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + s * L::kStageBytes;
          const uint32_t full_even = mapa_shared(full0 + 8 * s, 0);
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
          tma_load_2d_pair(sa, &maps.a, (t.k_block + kb) * kBK, t.a_row + (int)rank * 128, full_even);
          // B's K blocks are numbered as A's where both hold a stretch of K
          const int b_k = (p.by_rows ? kb : t.k_block + kb) * kBK, b_row = t.b_row + (int)rank * half;
          if (half == kMaxN / 2) {
            tma_load_2d_pair(sa + L::kABytes, &maps.b, b_k, b_row, full_even);
          } else {
            for (int i = 0; i < half; i += kBoxRows)
              tma_load_2d_pair(sa + L::kABytes + i * kBK, &maps.b16, b_k, b_row + i, full_even);
          }
          tma_load_2d_pair(sa + L::kSfaOff, &maps.sfa, 0, (int)(sfa + kb), full_even);
          tma_load_2d_pair(sa + L::kSfbOff, &maps.sfb, 0, (int)(t.b_atom + kb), full_even);
          if (second)
            tma_load_2d_pair(sa + L::kSfbOff + 512, &maps.sfb, 0, (int)(t.b_atom + p.b.atoms_k + kb),
                             full_even);
        }
      }
      // every slot's last release (the even CTA's commits) has arrived here
      for (uint32_t j = 0, jt = it; ok && j < (uint32_t)kStages; ++j, ++jt)
        ok = wait_bounded(empty0 + 8 * (jt % kStages), ((jt / kStages) & 1u) ^ 1u, abort_flag, err);
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
    for (int u = unit0; u < total && ok; u += unit_step) {
      const Tile t = find_tile(p, first, u);
      if (t.num_k == 0) continue;   // zeros, which the epilogue writes
      const uint32_t idesc = idesc_mxf8f6f4((uint32_t)p.a_format, (uint32_t)p.b_format, 256,
                                            (uint32_t)t.n, 0, 0);
      if (!wait_bounded_all(acce, (acc_it & 1u) ^ 1u, abort_flag, err)) break;
      tc_fence_after();
      for (int kb = 0; kb < t.num_k; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        if (!wait_bounded_all(full0 + 8 * s, ph, abort_flag, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          issue_block(ring + s * L::kStageBytes, tmem_base, tmem_base + kMaxN + L::kSfCols * s, idesc,
                      t.n > 128, kb == 0);
          mma_commit_pair_multicast(empty0 + 8 * s, kBoth);
          if (kb == t.num_k - 1) mma_commit_pair_multicast(accf, kBoth);
        }
        __syncwarp();
      }
      ++acc_it;
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
    // Warp w drains TMEM lane quarter w % 4 and rows of B [128 h, 128 h + 128)
    // with h = (w - 2) / 4, 32 at a time.
    const int quarter = warp & 3, h = (warp - 2) >> 2;
    const uint32_t acce_even = mapa_shared(acce, 0);
    uint32_t acc_it = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const Tile t = find_tile(p, first, u);
      Column<T> r[4];
      if (t.num_k > 0) {
        if (!wait_bounded_warp(accf, acc_it & 1u, abort_flag, err)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (128 * h + 32 * c < t.valid) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + 128 * h + 32 * c, v);
            tmem_ld_wait();
            r[c].take(v);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {   // the accumulator is free for the next tile
          if (rank == 0)
            mbar_arrive(acce);
          else
            mbar_arrive_cluster(acce_even);
        }
        ++acc_it;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) r[c].clear();
      }
      const int m = t.col + (int)rank * 128 + quarter * 32 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n0 = 128 * h + 32 * c;
        if (n0 < t.valid)
          r[c].store(static_cast<T *>(p.C), p.a_rows, t.c_row + n0, m, p.a_rows, t.valid - n0);
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

bool data_map(CUtensorMap *m, const Side &s, uint32_t box_rows) {
  return make_tmap_2d(m, s.data, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)s.row_bytes,
                      (uint64_t)s.rows, (uint64_t)s.row_bytes, kBK, box_rows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

// The scale atoms as a matrix with an atom a row.
bool scale_map(CUtensorMap *m, const Side &s, int64_t atoms) {
  return make_tmap_2d(m, s.scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128, (uint64_t)atoms, 512, 128, 1,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <typename T>
int run_product(const PairMaps &maps, const ProductArgs &a, int64_t most, cudaStream_t stream) {
  auto kernel = product_kernel<T>;
  static PerDeviceOnce setup;  // per instantiation: the pairs that fit at once, 0 on failure
  const int pairs = setup.get([&] {
    if (gemm::set_smem(kernel, Layout::kSmemBytes) != cudaSuccess) return 0;
    Launch q(2 * (sm_count() / 2), 1, kThreads, Layout::kSmemBytes, stream, 2);
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q.cfg) == cudaSuccess ? n : 0;
  });
  unsigned int *err = device_error_word();
  if (pairs < 1 || err == nullptr) return FP8Q_ERR_CUDA;
  const int grid = 2 * (int)std::min<int64_t>(most, pairs);
  log_line("launch experts product_kernel, %d groups, tile 256x256, grid %d in pairs", a.groups.count, grid);
  return Launch((unsigned)grid, 1, kThreads, Layout::kSmemBytes, stream, 2)
                     .run(kernel, maps, a, err) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

}  // namespace

int launch_product(const ProductArgs &a, int out_dtype, int64_t a_atoms, int64_t b_atoms,
                   cudaStream_t stream) {
  PairMaps maps;
  if (!data_map(&maps.a, a.a, 128) || !data_map(&maps.b, a.b, kMaxN / 2) ||
      !data_map(&maps.b16, a.b, kBoxRows) || !scale_map(&maps.sfa, a.a, a_atoms) ||
      !scale_map(&maps.sfb, a.b, b_atoms))
    return FP8Q_ERR_CUDA;
  // the most tiles that the groups can make
  const int64_t across = (a.a_rows + 255) / 256;
  const int64_t most =
      across * (a.by_rows ? std::min<int64_t>(a.groups.rows, a.groups.rows / kMaxN + a.groups.count)
                          : (int64_t)a.groups.count * ((a.b_rows + kMaxN - 1) / kMaxN));
  if (most > kMostTiles) return FP8Q_ERR_INVALID_ARG;
  return out_dtype == FP8Q_DT_BF16 ? run_product<__nv_bfloat16>(maps, a, most, stream)
                                   : run_product<float>(maps, a, most, stream);
}

}  // namespace experts
}  // namespace fp8q
