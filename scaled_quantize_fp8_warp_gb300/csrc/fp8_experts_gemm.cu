// The products of a layer of experts in MXFP8, per group e, on the tensor cores'
// own block scaling (tcgen05.mma kind::mxf8f6f4): scales go from shared into
// tensor memory ahead of each K block's MMAs, the whole contraction accumulates
// in fp32 in tensor memory.
//
// fprop, dgrad (C = B . A_e^T): a weight's rows are the MMA's M, 256 a tile, 128 in
// each CTA of a pair (cta_group::2); the group's rows, whose number the router
// decided, are its N, up to 256 and as few as 32.  So a group of a few rows costs
// MMAs and loads of 32 rows and not of 256, and groups may start anywhere.  A
// column of C comes out in every lane; a warp stores 32 neighbouring columns.
// wgrad (C_e = A_e . B_e^T): both sides are known on the host, the contraction is
// the group's.  A row of C comes out in every lane and leaves through shared
// memory by TMA, clipped at the weight's edges.
//
// Roles: one warp loads, one (of the even CTA) issues the MMAs, one finds the
// tiles ahead of both from the offsets, the others take the results out.  A tile's
// coordinates pass through a ring in shared memory: found by each role for
// itself they cost some 750 cycles of every tile.  Persistent, every grid-th tile,
// group after group, so that neighbours read the same weight.
//
// What bounds it: shared memory.  A K block of 128 moves 16 KB of A and n / 2 rows of
// B into each CTA and reads them once in MMAs of 2 n cycles, 256 + n cycles at 128
// bytes a cycle: 512 for n = 256, where the MMAs take 512 too, 384 for n = 128, where
// they take 256.  Captured, on a GPU that was idle: 16384 rows in one group, 2048 x
// 4096 83 us (3.3 PFLOP/s; MMAs alone 69); in 32 groups of unlike sizes 106 (2.6;
// loads alone 86, tensor pipe busy 67% of an SM's time there, and 12% of the time is
// before the first or behind the last tile of an SM), dgrad of them 115, to fp32 148;
// in 128 groups, 1024 x 4096 90 (its 537 MB of weights at the copy rate: 82).  wgrad of
// the 32 groups 148 us, 537 MB of results, to fp32 247; with 64 rows a group 90.
// After a second of them the power limit lowers the clock from 2070 to 1600 - 1950
// MHz: fprop 120, dgrad 126, wgrad 156.
//
// Tried, each against the kernel of its day (fprop of the 32 groups went from 116 to
// 112, 110 and 107 us, wgrad from 219 to 146 and 148): tiles 384 wide (two MMAs a step,
// five stages) 118 us where 256 took 112, and one token 24.5 for 18.3: fewer bytes of
// the weight are under way.  A's blocks called into L2 ahead: no gain.  Groups sorted
// by what a tile of theirs costs: 1% here, more lost elsewhere.  Scales copied a
// block ahead of their MMAs: 110 for 107.  wgrad by places of C_e instead of group by
// group: 229 for 219, DRAM reads 291 MB for 126.  Tiles of wgrad 128 wide with three
// accumulators: 161.  kRaster of 4 or 16: level.  Arriving at the even CTA's barrier
// with cluster-scope release: wgrad 219 us for 146.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp4_ptx.cuh"
#include "fp8_experts.h"
#include "fp8_experts_maps.h"
#include "fp8_experts_turns.h"
#include "fp8_pack8.cuh"
#include "fp8q_gemm_common.cuh"

namespace fp8q {
namespace experts {
namespace {

using namespace ptx;

constexpr int kRaster = 8;        // tiles of B visited together
constexpr int kTilesAhead = 8;    // tiles that are found ahead of their results
constexpr int kMostTiles = INT32_MAX / 2;   // of a launch
constexpr int kApart = INT32_MIN;   // in place of an offset that A and B do not share

struct PairMaps {
  CUtensorMap a, b[4], sfa, sfb;   // b: boxes of 128, 64, 32 and 16 rows
  CUtensorMap c;                   // wgrad: the results
};

// One tile: what of A, B and K it takes, and where its result goes.
struct __align__(16) Tile {
  int a_row, b_row;        // first rows of A and of B
  int k_block, num_k;      // K blocks; num_k < 0: A and B have other groups, the result is NaN
  int a_block, b_block;    // 128-row blocks of the scales of the first rows
  int n, valid;            // rows of B: as the MMA takes them (a multiple of 32), and those that count
  int across, along;       // first rows of the tile in the group's parts of A and B
  int64_t c_row;           // ROWS: row of C of the first row of B; else the group
};

// ROWS: groups own rows of C, which are B's rows and lie across the lanes
// (fprop, dgrad); otherwise C's rows are A's and lie along the lanes (wgrad).
// WIDE: rows of B per tile, 256 or 128.
template <typename T, bool ROWS, int WIDE>
struct Layout {
  static constexpr int kRowBlocks = WIDE / 128;
  static constexpr int kABytes = 128 * kBK, kBBytes = WIDE / 2 * kBK;
  static constexpr int kSfaOff = kABytes + kBBytes, kSfbOff = kSfaOff + 512;
  static constexpr int kStageBytes = (kSfbOff + kRowBlocks * 512 + 1023) / 1024 * 1024;
  // Tensor memory: accumulators, then a slot of scales per stage.  256 columns
  // leave no room for a second accumulator.
  static constexpr uint32_t kTmemCols = 512, kSfCols = 4 * (1 + kRowBlocks);
  static constexpr int kAcc = WIDE == 256 ? 1 : 3;
  // Epilogue warps: teams take tiles in turn, so that one team's stores go out
  // while the other waits for its tile.  In a team a warp has 32 lanes and
  // kChunks chunks of 32 rows of B; a lone accumulator is taken into registers
  // at once and released (bf16 only: fp32 results would not fit).
  static constexpr int kTeams = kAcc > 1 ? 2 : 1;
  static constexpr int kColumnGroups = kAcc > 1 ? 1 : 2;
  // Tile j takes accumulator j % kAcc and is announced on barrier j % kFull.  A
  // barrier is one team's alone and the team waits for each of its phases: a wait
  // names a phase by its parity, so one that is two phases early passes.
  static constexpr int kFull = kAcc * kTeams;
  static_assert(kFull % kTeams == 0 && kTilesAhead % kTeams == 0, "a barrier serves one team");
  static_assert(kAcc > 1 || sizeof(T) == 2, "a tile's results fit in registers");
  static constexpr int kTeamWarps = 4 * kColumnGroups;
  static constexpr int kEpilogueWarps = kTeams * kTeamWarps;
  static constexpr int kChunks = WIDE / 32 / kColumnGroups;
  static constexpr int kThreads = 32 * (3 + kEpilogueWarps);
  // Results along the lanes leave through shared memory, a chunk of 32 x 32 a warp
  // at a time: what staging takes, the ring lacks (wgrad.  Bf16, six stages as here:
  // 64 groups of 64 rows, 1024 x 2048 53.3 us, 16384 rows in 8, 2048 x 4096 93.4; 32 x 64
  // a warp and five stages 58.7 and 95.8; two places a warp and four 58.0 and 101.6).
  static constexpr int kPieceBytes = 1024 * (int)sizeof(T);
  static constexpr int kOutBytes = ROWS ? 0 : kEpilogueWarps * kPieceBytes;
  // the groups' offsets, and the first tile of each where it depends on them
  static constexpr int kGroupBytes = (ROWS ? 2 : 1) * (FP8Q_EXPERTS_MAX + 1) * 4;
  static constexpr int kOtherBytes = 16 + kTilesAhead * (int)sizeof(Tile) + kGroupBytes + 1024;
  static constexpr int kStages = (227 * 1024 - 512 - kOtherBytes - kOutBytes) / kStageBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kBarBytes = 8 * (2 * kStages + kFull + kAcc + 2 * kTilesAhead + 2) / 16 * 16;
  static constexpr int kSmemBytes = kRingBytes + kOutBytes + kBarBytes + kOtherBytes;
  static_assert(kSmemBytes <= 227 * 1024, "the ring fits in shared memory");
  static_assert(WIDE * kAcc + kSfCols * kStages <= kTmemCols, "scale slots fit in tensor memory");
};

// Tiles along B for so many of its rows, and across A.
template <int WIDE>
__device__ __forceinline__ int tiles_along(int rows) { return (rows + WIDE - 1) / WIDE; }
__device__ __forceinline__ int tiles_across(const ProductArgs &p) { return (p.a_rows + 255) / 256; }

// Where every group's tiles start in the numbering of all, by one warp (ROWS).
template <int WIDE>
__device__ __forceinline__ void number_tiles(const ProductArgs &p, const int32_t *offsets, int *first) {
  const int lane = threadIdx.x & 31, E = p.groups.count;
  long long done = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    long long n = 0;
    if (e0 + lane < E)
      n = (long long)tiles_along<WIDE>(group_rows(p.groups, offsets, e0 + lane).y) * tiles_across(p);
    long long sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long other = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += other;
    }
    if (e0 + lane < E) first[e0 + lane] = (int)min(done + sum - n, (long long)kMostTiles);
    done += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  // more than the host allows for come from offsets that are no offsets: nothing is done
  if (lane == 0) first[E] = done <= kMostTiles ? (int)done : 0;
}

// The tiles of one CTA pair, in their order: every `step`-th of all, group after
// group; next() is false behind the last.
template <bool ROWS, int WIDE>
struct Tiles {
  const ProductArgs &p;
  const int32_t *offsets;
  const int *first;
  int u, step;
  int e = -1, row, rows;       // the group, its first row and its rows
  int block, along, each, more;
  bool apart = false;          // the group begins or ends elsewhere in A
  __device__ __forceinline__ Tiles(const ProductArgs &args, const int32_t *group_offsets,
                                   const int *first_tiles, int pair, int pairs)
      : p(args), offsets(group_offsets), first(first_tiles), u(pair), step(pairs) {}
  __device__ __forceinline__ int first_of(int group) const {
    return ROWS ? first[group] : group * (tiles_along<WIDE>(p.b_rows) * tiles_across(p));
  }
  __device__ __forceinline__ bool next(Tile &t) {
    if (u >= first_of(p.groups.count)) return false;
    if (e < 0 || u >= first_of(e + 1)) {
      if (ROWS) {
        int lo = e + 1, hi = p.groups.count;   // first[lo] <= u < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (first[mid] <= u)
            lo = mid;
          else
            hi = mid;
        }
        e = lo;
      } else {
        e = u / first_of(1);
      }
      const int2 group = group_rows(p.groups, offsets, e);
      if (!ROWS && p.a_offsets != nullptr) apart = offsets[e] == kApart || offsets[e + 1] == kApart;
      row = group.x;
      rows = group.y;
      block = first_block(p.groups, e, row);
      const int n = ROWS ? rows : p.b_rows, blocks = (n + 127) / 128;
      along = tiles_along<WIDE>(n);
      each = blocks / along;   // whole 128-row blocks, as evenly as they go
      more = blocks - each * along;
    }
    int bt, at;
    gemm::tile_coords(u - first_of(e), along, tiles_across(p), bt, at, kRaster, 0);
    const int b0 = bt * each + min(bt, more), b1 = b0 + each + (bt < more);
    t.across = at * 256;
    t.along = b0 * 128;
    t.valid = min(b1 * 128, ROWS ? rows : p.b_rows) - t.along;
    t.n = (t.valid + 31) / 32 * 32;
    if (ROWS) {
      t.a_row = p.a_row * e + t.across;
      t.b_row = row + t.along;
      t.k_block = p.a_k * e;
      t.num_k = (p.k + kBK - 1) / kBK;
      t.a_block = p.a_block * e + 2 * at;
      t.b_block = block + b0;
      t.c_row = row + t.along;
    } else {
      t.a_row = t.across;
      t.b_row = t.along;
      t.k_block = block;
      t.num_k = apart ? -1 : (rows + kBK - 1) / kBK;
      t.a_block = 2 * at;
      t.b_block = b0;
      t.c_row = e;
    }
    u += step;
    return true;
  }
};

// One K block in the ring slot at `sa`, by one elected thread: scales into
// tensor memory at sf, then four MMAs of K = 32.
template <typename L>
__device__ __forceinline__ void issue_block(uint32_t sa, uint32_t d_tmem, uint32_t sf, uint32_t idesc,
                                            bool second, bool first) {
  const uint64_t atom = sdesc_plain(sa + L::kSfaOff, 128);   // + 32 per atom
  tmem_cp_32x128b_x4_pair(sf, atom);
  tmem_cp_32x128b_x4_pair(sf + 4, atom + 32);
  if (L::kRowBlocks > 1 && second) tmem_cp_32x128b_x4_pair(sf + 8, atom + 64);
  const uint64_t ad = sdesc_k(sa, gemm::kSwzSBO, gemm::kSwzMode);
  const uint64_t bd = sdesc_k(sa + L::kABytes, gemm::kSwzSBO, gemm::kSwzMode);
#pragma unroll
  for (int k = 0; k < 4; ++k)   // step k uses byte k of each scale word
    mma_mxf8f6f4_pair(d_tmem, ad + 2 * k, bd + 2 * k, idesc | ((uint32_t)k << 29) | ((uint32_t)k << 4),
                      sf, sf + 4, (!first || k > 0) ? 1u : 0u);
}

// `rows` rows of B from `row` on, a multiple of 16, in as few boxes as there are.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap (&maps)[4], int k, int row,
                                          int rows, uint32_t full) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (rows & (128 >> i)) {
      tma_load_2d_pair(dst, &maps[i], k, row, full);
      dst += (128 >> i) * kBK;
      row += 128 >> i;
    }
}

// Results of one row of A and 32 rows of B, as they are kept for storing:
// bf16 ones two to a register.
template <typename T>
struct Chunk {
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
  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int j = 0; j < kRegs; ++j) r[j] = sizeof(T) == 4 ? 0x7FC00000u : 0x7FC07FC0u;
  }
  // Into this lane's row of 64 or 128 bytes, as swizzling of that width has them.
  __device__ __forceinline__ void stage(uint32_t row) const {
#pragma unroll
    for (int c = 0; c < kRegs / 4; ++c)
      st_shared_16(row + (((uint32_t)c << 4) ^ (row >> 3 & 4u * kRegs - 16u)), r[4 * c], r[4 * c + 1],
                   r[4 * c + 2], r[4 * c + 3]);
  }
  // Into column m of C from row c_row on, `count` rows of it; lanes hold
  // neighbouring columns.
  __device__ __forceinline__ void store_column(T *C, int64_t ld, int64_t c_row, int m, int columns,
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

template <typename T, bool ROWS, int WIDE>
__global__ void __launch_bounds__(Layout<T, ROWS, WIDE>::kThreads, 1)
    product_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ ProductArgs p,
                   unsigned int *err) {
  using L = Layout<T, ROWS, WIDE>;
  constexpr int kStages = L::kStages;
  constexpr uint16_t kBoth = 3;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + L::kRingBytes + L::kOutBytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
  const uint32_t accf0 = bars + 8 * (2 * kStages), acce0 = accf0 + 8 * L::kFull;
  const uint32_t tilef0 = acce0 + 8 * L::kAcc, tilee0 = tilef0 + 8 * kTilesAhead;
  const uint32_t drain = tilee0 + 8 * kTilesAhead;
  const uint32_t slot = bars + L::kBarBytes;
  uint8_t *slot_ptr = smem_raw + (slot - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);
  Tile *tile_ring = reinterpret_cast<Tile *>(slot_ptr + 16);
  int32_t *offsets = reinterpret_cast<int32_t *>(tile_ring + kTilesAhead);
  int *first = offsets + FP8Q_EXPERTS_MAX + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: issues the pair's MMAs
  cluster_arrive_any();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < L::kFull; ++i) mbar_init(accf0 + 8 * i, 1);
    for (int i = 0; i < L::kAcc; ++i) mbar_init(acce0 + 8 * i, 2 * L::kTeamWarps);
    for (int i = 0; i < kTilesAhead; ++i) {   // read by the loading warp, in the even CTA the
      mbar_init(tilef0 + 8 * i, 1);           // issuing one, and a team of the epilogue
      mbar_init(tilee0 + 8 * i, (rank == 0 ? 2 : 1) + L::kTeamWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tmap(&maps.a);
    for (int i = 0; i < 4; ++i) prefetch_tmap(&maps.b[i]);
    prefetch_tmap(&maps.sfa);
    prefetch_tmap(&maps.sfb);
  }
  if (warp == 1) {
    tmem_alloc_pair(slot, L::kTmemCols);
    tmem_relinquish_pair();
  }
  follow_previous();
  allow_next();
  if (warp >= 2) {   // the epilogue's warps fetch the offsets
    if (p.groups.offsets != nullptr)
      for (int e = threadIdx.x - 64; e <= p.groups.count; e += 32 * L::kEpilogueWarps)
        if (warp < 2 + L::kEpilogueWarps) {
          const int32_t at = row_of(p.groups, p.groups.offsets[e]);
          offsets[e] = !ROWS && p.a_offsets != nullptr && row_of(p.groups, p.a_offsets[e]) != at ? kApart : at;
        }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);
  cluster_wait_any();   // the peer runs: its shared memory may be written
  if (warp == 1 && lane == 0) st_shared_cluster_u32(mapa_shared(slot + 8, rank ^ 1u), tmem_base);
  if (ROWS && warp == 2) number_tiles<WIDE>(p, offsets, first);
  __syncthreads();
  cluster_sync_any();
  // One allocation serves the pair: both CTAs must hold the same address.
  // Otherwise neither does any work (a symmetric decision, no waiting).
  const bool paired = *reinterpret_cast<volatile uint32_t *>(slot_ptr + 8) == tmem_base;
  if (!paired && threadIdx.x == 0) atomicOr(err, 4u);

  // Tile j of this CTA, by one thread that arrives for its warp, or by a
  // converged warp; false where there is none or the CTA aborts.
  const auto take_tile = [&](int j, bool warp_wide, Tile &t) {
    const int i = j % kTilesAhead;
    const uint32_t phase = (uint32_t)(j / kTilesAhead) & 1u;
    const bool ok = warp_wide ? wait_bounded_all(tilef0 + 8 * i, phase, abort_flag, err)
                              : wait_bounded(tilef0 + 8 * i, phase, abort_flag, err);
    if (!ok) return false;
    t = tile_ring[i];
    if (warp_wide) __syncwarp();
    if (!warp_wide || lane == 0) mbar_arrive(tilee0 + 8 * i);
    return t.valid > 0;
  };

  if (!paired) {
  } else if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      const int a_blocks = (p.a_rows + 127) / 128;   // 128-row blocks of a group's A
      Tile t;
      for (int j = 0; ok && take_tile(j, false, t); ++j) {
        // past the last block of A (odd count): the even CTA's scales again, nothing is stored
        const int a_block = t.a_block + (t.across / 128 + (int)rank < a_blocks ? (int)rank : 0);
        const int half = t.n / 2, b_row = t.b_row + (int)rank * half;   // this CTA's half of B's rows
        const uint32_t bytes = L::kABytes + (uint32_t)half * kBK + 512u * (1 + L::kRowBlocks);
        for (int kb = 0; kb < t.num_k; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + s * L::kStageBytes;
          const uint32_t full_even = mapa_shared(full0 + 8 * s, 0);
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
          // ROWS: B's contraction is its own, A's may be a stretch of a longer one
          const int a_k = t.k_block + kb, b_k = ROWS ? kb : a_k;
          tma_load_2d_pair(sa, &maps.a, a_k * kBK, t.a_row + (int)rank * 128, full_even);
          load_rows(sa + L::kABytes, maps.b, b_k * kBK, b_row, half, full_even);
          tma_load_2d_pair(sa + L::kSfaOff, &maps.sfa, a_k * 128, a_block, full_even);
          // blocks past the group's are another's or zeros; no MMA reads them
          tma_load_2d_pair(sa + L::kSfbOff, &maps.sfb, b_k * 128, t.b_block, full_even);
        }
      }
      // every slot's last release (the even CTA's commits) has arrived here
      ok = ok && !*abort_flag;
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
    uint32_t it = 0;
    bool ok = true;
    Tile t;
    int j = 0;
    for (; ok && take_tile(j, true, t); ++j) {
      const uint32_t idesc = idesc_mxf8f6f4((uint32_t)p.a_format, (uint32_t)p.b_format, 256,
                                            (uint32_t)t.n, 0, 0);
      const uint32_t acc = accumulator_of<L::kAcc>(j), turn = turn_of<L::kAcc>(j);
      const uint32_t accf = accf0 + 8 * ((uint32_t)j % L::kFull);
      ok = wait_bounded_all(acce0 + 8 * acc, (turn & 1u) ^ 1u, abort_flag, err);
      if (!ok) break;
      tc_fence_after();
      // an empty group's tile takes its turn too; the epilogue writes zeros (or NaN)
      if (!ROWS && t.num_k <= 0) {
        if (elect_one()) mma_commit_pair_multicast(accf, kBoth);
        __syncwarp();
      }
      for (int kb = 0; kb < t.num_k; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        if (!wait_bounded_all(full0 + 8 * s, ph, abort_flag, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          issue_block<L>(ring + s * L::kStageBytes, tmem_base + WIDE * acc,
                         tmem_base + WIDE * L::kAcc + L::kSfCols * s, idesc, t.n > 128, kb == 0);
          mma_commit_pair_multicast(empty0 + 8 * s, kBoth);
          if (kb == t.num_k - 1) mma_commit_pair_multicast(accf, kBoth);
        }
        __syncwarp();
      }
    }
    // The odd CTA's last releases land in this CTA's shared memory, and the barrier
    // at the end orders none of them: they are waited for here.  They were sent
    // before the last results' stores, so this waits for no store.
    if (ok)
      settle<L::kAcc>((uint32_t)j, [&](uint32_t a, uint32_t turn) {
        return wait_bounded_all(acce0 + 8 * a, turn & 1u, abort_flag, err);
      });
    if (elect_one()) {
      mma_commit_pair(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 200000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
  } else if (warp == 2 + L::kEpilogueWarps) {
    // finds the tiles ahead of the others
    Tiles<ROWS, WIDE> tiles(p, offsets, first, blockIdx.x / 2, gridDim.x / 2);
    for (int j = 0, ends = 0; ends < L::kTeams; ++j) {
      Tile t;
      if (ends > 0 || !tiles.next(t)) {
        t.valid = 0;   // behind the last tile: one for each team
        ++ends;
      }
      const int i = j % kTilesAhead;
      if (!wait_bounded_all(tilee0 + 8 * i, ((uint32_t)(j / kTilesAhead) & 1u) ^ 1u, abort_flag, err)) break;
      if (lane == 0) {
        tile_ring[i] = t;
        mbar_arrive(tilef0 + 8 * i);
      }
      __syncwarp();
    }
  } else {
    // A warp of a team drains TMEM lane quarter w % 4 and the kChunks chunks of
    // 32 rows of B that are its.
    const int team = (warp - 2) / L::kTeamWarps;
    const int quarter = warp & 3, h = (warp - 2) % L::kTeamWarps >> 2;
    const uint32_t acce_even = mapa_shared(acce0, 0);
    const uint32_t out = ring + L::kRingBytes + (warp - 2) * L::kPieceBytes;
    // chunks alternate between warps (ROWS: few rows are shared by all) or follow one another
    const auto chunk_at = [&](int c) { return 32 * (ROWS ? L::kColumnGroups * c + h : L::kChunks * h + c); };
    Tile t;
    for (int j = team; take_tile(j, true, t); j += L::kTeams) {
      const uint32_t acc = accumulator_of<L::kAcc>(j);
      const uint32_t from = tmem_base + ((uint32_t)(quarter * 32) << 16) + WIDE * acc;
      if (!wait_bounded_warp(accf0 + 8 * ((uint32_t)j % L::kFull), ((uint32_t)j / L::kFull) & 1u,
                             abort_flag, err))
        break;
      tc_fence_after();
      const auto release = [&] {   // the accumulator is free for another tile
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0)
            mbar_arrive(acce0 + 8 * acc);
          else
            mbar_arrive_peer(acce_even + 8 * acc);
        }
      };
      const int m = t.across + (int)rank * 128 + quarter * 32;   // first row of the group's A
      // kPiece chunks are loaded at once
      constexpr int kPiece = ROWS ? 2 : 4 / (int)sizeof(T);
      Chunk<T> r[L::kAcc > 1 ? kPiece : L::kChunks];
      const auto load = [&](Chunk<T> *to, int c) {
        uint32_t x[kPiece][32];
        if (ROWS || t.num_k > 0) {
          // a piece's store leaves lanes behind (those past the columns, the one that
          // issues TMA stores), and tcgen05.ld is the whole warp's
          if (L::kAcc > 1) __syncwarp();
#pragma unroll
          for (int k = 0; k < kPiece; ++k)
            if (chunk_at(c + k) < t.valid) tmem_ld_32x32b_x32(from + chunk_at(c + k), x[k]);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < kPiece; ++k) to[k].take(x[k]);
        } else {
#pragma unroll
          for (int k = 0; k < kPiece; ++k) to[k].clear();
          if (t.num_k < 0) {
            __syncwarp();   // a branch: as selects it costs every tile (151 us for 148)
#pragma unroll
            for (int k = 0; k < kPiece; ++k) to[k].poison();
          }
        }
      };
      const auto store = [&](const Chunk<T> *of, int c) {
        if constexpr (ROWS) {
#pragma unroll
          for (int k = 0; k < kPiece; ++k) {
            const int n0 = chunk_at(c + k);
            if (n0 < t.valid)
              of[k].store_column(static_cast<T *>(p.C), p.a_rows, t.c_row + n0, m + lane, p.a_rows,
                                 t.valid - n0);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kPiece; ++k) {
            const int n0 = chunk_at(c + k);
            if (n0 >= t.valid || m >= p.a_rows) return;
            if (lane == 0) bulk_wait_read();   // the piece before has left
            __syncwarp();
            of[k].stage(out + lane * (32 * sizeof(T)));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {   // rows and columns past the weight are not written
              tma_store_3d(&maps.c, out, t.along + n0, m, (int)t.c_row);
              bulk_commit();
            }
          }
        }
      };
      if constexpr (L::kAcc > 1) {
#pragma unroll
        for (int c = 0; c < L::kChunks; c += kPiece) {
          load(r, c);
          if (c + kPiece >= L::kChunks) release();
          store(r, c);
        }
      } else {
#pragma unroll
        for (int c = 0; c < L::kChunks; c += kPiece) load(r + c, c);
        release();
#pragma unroll
        for (int c = 0; c < L::kChunks; c += kPiece) store(r + c, c);
      }
    }
    if (!ROWS && lane == 0) bulk_wait();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive_any();
  // Neither CTA leaves while the other may still signal it: what was sent has been
  // waited for on its barrier (copies and commits by the loading warp and the
  // epilogue, releases by the issuing warp), this one counts CTAs only.
  cluster_wait_any();
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem_base, L::kTmemCols);
}

template <typename T, bool ROWS, int WIDE>
int run_product(const ProductArgs &a, int64_t a_atoms, int64_t b_atoms, cudaStream_t stream) {
  using L = Layout<T, ROWS, WIDE>;
  PairMaps maps;
  bool ok = data_map(&maps.a, a.a, 128) && scale_map(&maps.sfa, a.a, a_atoms, 1) &&
            scale_map(&maps.sfb, a.b, b_atoms, L::kRowBlocks);
  for (int i = 0; i < 4; ++i) ok = ok && data_map(&maps.b[i], a.b, 128u >> i);
  const uint64_t size = sizeof(T);
  if (!ROWS)
    ok = ok && make_tmap_3d(&maps.c, a.C, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                            (uint64_t)a.b_rows, (uint64_t)a.a_rows, (uint64_t)a.groups.count, a.b_rows * size,
                            a.a_rows * (a.b_rows * size), 32, 32, sizeof(T) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return FP8Q_ERR_CUDA;
  // the most tiles that the groups can make
  const int64_t along = ROWS ? std::min<int64_t>(a.groups.rows, a.groups.rows / WIDE + a.groups.count)
                             : (int64_t)a.groups.count * ((a.b_rows + WIDE - 1) / WIDE);
  const int64_t most = along * ((a.a_rows + 255) / 256);
  if (most > kMostTiles) return FP8Q_ERR_INVALID_ARG;
  auto kernel = product_kernel<T, ROWS, WIDE>;
  static PerDeviceOnce setup;  // per instantiation: the pairs that fit at once, 0 on failure
  const int pairs = setup.get([&] {
    if (gemm::set_smem(kernel, L::kSmemBytes) != cudaSuccess) return 0;
    Launch q(2 * (sm_count() / 2), 1, L::kThreads, L::kSmemBytes, stream, 2);
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q.cfg) == cudaSuccess ? n : 0;
  });
  unsigned int *err = device_error_word();
  if (pairs < 1 || err == nullptr) return FP8Q_ERR_CUDA;
  const int grid = 2 * (int)std::min<int64_t>(most, pairs);
  log_line("launch experts product_kernel, %d groups, tile 256x%d, grid %d in pairs", a.groups.count,
           WIDE, grid);
  return Launch((unsigned)grid, 1, L::kThreads, L::kSmemBytes, stream, 2)
                     .run(kernel, maps, a, err) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

}  // namespace

int launch_product(const ProductArgs &a, int out_dtype, int64_t a_atoms, int64_t b_atoms,
                   cudaStream_t stream) {
  const bool bf16 = out_dtype == FP8Q_DT_BF16;
  if (!a.by_rows)
    return bf16 ? run_product<__nv_bfloat16, false, 256>(a, a_atoms, b_atoms, stream)
                : run_product<float, false, 128>(a, a_atoms, b_atoms, stream);
  const int split = split_for(a);
  if (split > 0) return launch_split(a, split, out_dtype, a_atoms, b_atoms, stream);
  // Tiles 128 wide, which have a deeper ring and three accumulators, up to 96 rows
  // a group on average, as far as the host knows (rows behind the last group count):
  // 64 equal groups, 1024 x 4096, 1024 rows 49.6 us and 52.4 with
  // 256-wide tiles; groups of unlike sizes, 4000 rows in 50, 2048 x 1024, 25.2 and
  // 26.2, but 8192 in 64, 1024 x 4096, 56.5 and 54.6.
  if (bf16 && a.groups.rows > 96 * (int64_t)a.groups.count)
    return run_product<__nv_bfloat16, true, 256>(a, a_atoms, b_atoms, stream);
  return bf16 ? run_product<__nv_bfloat16, true, 128>(a, a_atoms, b_atoms, stream)
              : run_product<float, true, 128>(a, a_atoms, b_atoms, stream);
}

}  // namespace experts
}  // namespace fp8q
