// The products of a layer of experts for few rows, C_e = B_e . A_e^T with B's rows
// in groups (fprop and dgrad), where reading the weights once is the work and
// the pairs' 256 x 256 tiles would leave most SMs idle.
//
// As in the kernel on CTA pairs a tile's weight rows are the MMA's M, here 128 of
// them in one CTA, and the group's rows its N, as few as 16.  The contraction of
// a tile is split over the CTAs of a cluster, which stream their parts of the
// weight at once; their partial sums meet in distributed shared memory and are
// added in the order of the ranks, so results do not depend on timing.
//
// Two CTAs share an SM, with 256 of its 512 columns of tensor memory each.  (No
// third one fits their 112 KB of shared memory, nor any other kernel of this
// library that allocates tensor memory: an allocation never waits for a CTA
// that waits for this one's cluster.)
//
// What bounds it: latency.  In a graph, each call with other weights so that they
// come from HBM: 1 row, 1024 x 4096 5.8 us and 4096 x 4096 6.8 (bytes at the measured
// copy rate 0.6 and 2.5), 32 rows, 2048 x 4096 7.2; the kernel on pairs takes 10.8, 10.6
// and 10.7.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_launch.cuh"
#include "fp4_ptx.cuh"
#include "fp8_experts.h"
#include "fp8_experts_maps.h"
#include "fp8_pack8.cuh"
#include "fp8q_gemm_common.cuh"

namespace fp8q {
namespace experts {
namespace {

using namespace ptx;

constexpr int kEpilogueWarps = 4;
constexpr int kThreads = 32 * (2 + kEpilogueWarps);
constexpr int kWide = 128;                 // rows of B per tile at most
constexpr int kMaxStages = 5;
constexpr int kMaxSplit = 8;               // CTAs of a cluster (the portable limit)
constexpr int kSmemBytes = 112 * 1024;     // two CTAs on an SM, never three
constexpr int kFixedBytes = 1024 /* alignment */ + 8 * (2 * kMaxStages + 2) + 48 +
                            (FP8Q_EXPERTS_MAX + 1) * 4;
constexpr uint32_t kTmemCols = 256, kSfCols = 8;
constexpr int kSfaOff = 128 * kBK, kSfbOff = kSfaOff + 512, kBOff = kSfbOff + 512;

struct SplitMaps {
  CUtensorMap a, b[4], sfa, sfb;   // b: boxes of 128, 64, 32 and 16 rows
};

struct SplitArgs {
  ProductArgs p;
  int split, stages, stage_bytes;
  unsigned int *err;
};

// What a cluster works on.
struct Found {
  int e, row, rows;   // the group, its first row and rows; e < 0: nothing
  int local;          // tile in the group
};

// Tile u of all, by one warp from the offsets in shared memory: along a group
// whole 128-row blocks, and `across` tiles of A for each.
__device__ __forceinline__ Found find(const Groups &g, const int32_t *offsets, int across, int u) {
  const int lane = threadIdx.x & 31;
  long long done = 0;
  Found f{-1, 0, 0, 0};
  for (int e0 = 0; e0 < g.count; e0 += 32) {
    int2 group = make_int2(0, 0);
    if (e0 + lane < g.count) group = group_rows(g, offsets, e0 + lane);
    const long long n = (long long)((group.y + kWide - 1) / kWide) * across;
    long long sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long other = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += other;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, done + sum > u);
    if (past != 0) {   // the first group that ends behind u
      const int from = __ffs(past) - 1;
      f.e = e0 + from;
      f.row = __shfl_sync(0xFFFFFFFFu, group.x, from);
      f.rows = __shfl_sync(0xFFFFFFFFu, group.y, from);
      f.local = (int)(u - (done + __shfl_sync(0xFFFFFFFFu, sum - n, from)));
      return f;
    }
    done += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return f;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    split_product_kernel(const __grid_constant__ SplitMaps maps, const __grid_constant__ SplitArgs args) {
  const ProductArgs &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + args.stages * args.stage_bytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kMaxStages;
  const uint32_t accf = bars + 8 * (2 * kMaxStages), drain = accf + 8;
  uint8_t *slot_ptr = smem_raw + (drain + 8 - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);
  Found *found = reinterpret_cast<Found *>(slot_ptr + 16);
  int32_t *offsets = reinterpret_cast<int32_t *>(slot_ptr + 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < args.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
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
    tmem_alloc(smem_u32(slot_ptr), kTmemCols);
    tmem_relinquish();
  }
  follow_previous();
  allow_next();
  if (p.groups.offsets != nullptr)
    for (int e = threadIdx.x; e <= p.groups.count; e += kThreads) offsets[e] = p.groups.offsets[e];
  __syncthreads();
  const int across = (p.a_rows + 127) / 128;
  if (warp == 2) {
    const Found f = find(p.groups, offsets, across, (int)(blockIdx.x / (unsigned)args.split));
    if (lane == 0) *found = f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);
  const Found f = *found;
  const bool work = f.e >= 0;   // the same for the whole cluster

  const int bt = f.local / across, at = f.local - bt * across;   // blocks along B, across A
  const int valid = min(kWide, f.rows - bt * kWide), n = (valid + 15) / 16 * 16;
  const int num_k = work ? (p.k + kBK - 1) / kBK : 0;
  const int kb0 = (int)((int64_t)num_k * rank / args.split);
  const int count = (int)((int64_t)num_k * (rank + 1) / args.split) - kb0;   // K blocks of this CTA
  const uint32_t stages = (uint32_t)args.stages;

  if (!work) {
  } else if (warp == 0) {
    if (elect_one()) {
      const int a_row = p.a_row * f.e + at * 128, a_k = p.a_k * f.e, a_block = p.a_block * f.e + at;
      const int b_row = f.row + bt * kWide, b_block = first_block(p.groups, f.e, f.row) + bt;
      const uint32_t bytes = 128 * kBK + (uint32_t)n * kBK + 1024u;
      bool ok = true;
      int i = 0;
      for (; i < count && ok; ++i) {
        const uint32_t s = (uint32_t)i % stages, ph = ((uint32_t)i / stages) & 1u;
        if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, args.err)) {
          ok = false;
          break;
        }
        const uint32_t sa = ring + s * args.stage_bytes, full = full0 + 8 * s;
        mbar_arrive_expect_tx(full, bytes);
        tma_load_2d(sa, &maps.a, (a_k + kb0 + i) * kBK, a_row, full);
        tma_load_2d(sa + kSfaOff, &maps.sfa, (a_k + kb0 + i) * 128, a_block, full);
        uint32_t dst = sa + kBOff;
        int row = b_row;
#pragma unroll
        for (int m = 0; m < 4; ++m)   // n rows of B in as few boxes as there are
          if (n & (128 >> m)) {
            tma_load_2d(dst, &maps.b[m], (kb0 + i) * kBK, row, full);
            dst += (128 >> m) * kBK;
            row += 128 >> m;
          }
        tma_load_2d(sa + kSfbOff, &maps.sfb, (kb0 + i) * 128, b_block, full);
      }
      // copies that nobody may wait for any more land before the CTA goes on
      if (!ok)
        for (int j = max(0, i - args.stages); j < i; ++j) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full0 + 8 * ((uint32_t)j % stages), ((uint32_t)j / stages) & 1u) &&
                 globaltimer_ns() - t0 < 200000000ull) {
          }
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_mxf8f6f4((uint32_t)p.a_format, (uint32_t)p.b_format, 128, (uint32_t)n, 0, 0);
    for (int i = 0; i < count; ++i) {
      const uint32_t s = (uint32_t)i % stages;
      if (!wait_bounded_all(full0 + 8 * s, ((uint32_t)i / stages) & 1u, abort_flag, args.err)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = ring + s * args.stage_bytes, sf = tmem_base + kWide + kSfCols * s;
        tmem_cp_32x128b_x4(sf, sdesc_plain(sa + kSfaOff, 128));
        tmem_cp_32x128b_x4(sf + 4, sdesc_plain(sa + kSfbOff, 128));
        const uint64_t ad = sdesc_k(sa, gemm::kSwzSBO, gemm::kSwzMode);
        const uint64_t bd = sdesc_k(sa + kBOff, gemm::kSwzSBO, gemm::kSwzMode);
#pragma unroll
        for (int k = 0; k < 4; ++k)   // step k uses byte k of each scale word
          mma_mxf8f6f4(tmem_base, ad + 2 * k, bd + 2 * k,
                       idesc | ((uint32_t)k << 29) | ((uint32_t)k << 4), sf, sf + 4,
                       (i > 0 || k > 0) ? 1u : 0u);
        mma_commit(empty0 + 8 * s);
        if (i == count - 1) mma_commit(accf);
      }
      __syncwarp();
    }
    if (elect_one()) gemm::drain_mma(drain, abort_flag);
    __syncwarp();
  } else {
    // The sums of this CTA's part of K, [row of B][128 columns of C] in fp32,
    // where the ring was: its last copies have been read.
    const int quarter = warp & 3;
    const bool ok = wait_bounded_warp(accf, 0, abort_flag, args.err);
    tc_fence_after();
    for (int c = 0; ok && c < valid; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + c, v);
      tmem_ld_wait();
      const uint32_t to = ring + (uint32_t)(c * 128 + quarter * 32 + lane) * 4;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < valid)
          asm volatile("st.shared::cta.b32 [%0], %1;" ::"r"(to + 512 * j), "r"(v[j]) : "memory");
    }
  }
  __syncwarp();
  cluster_sync_any();   // all sums are there
  if (work && warp >= 2 && !*abort_flag) {
    // Each rank adds and stores its share of the rows, four columns a thread
    // and a row a warp.
    const int r0 = valid * (int)rank / args.split, r1 = valid * ((int)rank + 1) / args.split;
    const int m = at * 128 + 4 * lane;
    for (int r = r0 + warp - 2; r < r1; r += kEpilogueWarps) {
      const uint32_t at_row = ring + (uint32_t)(r * 128 + 4 * lane) * 4;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = 0; k < args.split; ++k) {
        const float4 v = ld_shared_cluster_f4(mapa_shared(at_row, (uint32_t)k));
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
      if (m >= p.a_rows) continue;   // a_rows % 16 == 0: all four or none
      T *to = static_cast<T *>(p.C) + (int64_t)(f.row + bt * kWide + r) * p.a_rows + m;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack8::bf16x2(sum.x, sum.y), pack8::bf16x2(sum.z, sum.w));
      else
        *reinterpret_cast<float4 *>(to) = sum;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive_any();
  cluster_wait_any();   // no CTA leaves while another may read its sums
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
}

// Clusters of `split` CTAs that run at once on the current device.
template <typename T>
int clusters_at_once(int split) {
  static PerDeviceOnce setup[kMaxSplit + 1];
  auto kernel = split_product_kernel<T>;
  return setup[split].get([&] {
    if (gemm::set_smem(kernel, kSmemBytes) != cudaSuccess) return 0;
    Launch q((unsigned)(2 * sm_count() / split * split), 1, kThreads, kSmemBytes, nullptr, split);
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q.cfg) == cudaSuccess ? n : 0;
  });
}

// The most tiles that the groups can make, each of fewer rows than a tile has.
int64_t most_tiles(const ProductArgs &a) {
  return std::min<int64_t>(a.groups.rows, a.groups.count) * ((a.a_rows + 127) / 128);
}

template <typename T>
int run_split(const SplitMaps &maps, const SplitArgs &args, cudaStream_t stream) {
  if (clusters_at_once<T>(args.split) < 1) return FP8Q_ERR_CUDA;
  const unsigned grid = (unsigned)(most_tiles(args.p) * args.split);
  log_line("launch experts split_product_kernel, %d groups, K over %d CTAs, grid %u", args.p.groups.count,
           args.split, grid);
  return Launch(grid, 1, kThreads, kSmemBytes, stream, args.split)
                     .run(split_product_kernel<T>, maps, args) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

}  // namespace

// Where the clusters of all tiles run at once, with four K blocks a CTA at
// least, four or eight CTAs to a tile and fewer than 128 rows in all.  Both sides
// of the line, captured, weights from HBM, this kernel and the pairs': 1 row, 1024
// x 4096 5.8 us and 10.8; 16 rows in 4 groups, 1024 x 2048 5.5 and 7.7; 100 rows in
// one, 2048 x 4096 9.4 and 11.8; but 128 rows, 4096 x 4096 14.9 and 11.9; and over two
// CTAs 13 rows in 12 groups, 1008 x 2000 9.6 and 8.9, 8 in 8, 2048 x 4096 15.8 and 15.3.
int split_for(const ProductArgs &a) {
  if (a.groups.rows >= kWide) return 0;
  const int64_t tiles = most_tiles(a), num_k = (a.k + kBK - 1) / kBK;
  for (int split = kMaxSplit; split >= 4; split /= 2)
    if (num_k >= 4 * split && tiles <= clusters_at_once<__nv_bfloat16>(split)) return split;
  return 0;
}

int launch_split(const ProductArgs &a, int split, int out_dtype, int64_t a_atoms, int64_t b_atoms,
                 cudaStream_t stream) {
  SplitMaps maps;
  bool ok = data_map(&maps.a, a.a, 128) && scale_map(&maps.sfa, a.a, a_atoms, 1) &&
            scale_map(&maps.sfb, a.b, b_atoms, 1);
  for (int i = 0; i < 4; ++i) ok = ok && data_map(&maps.b[i], a.b, 128u >> i);
  SplitArgs args{};
  args.p = a;
  args.split = split;
  const int rows = (a.groups.rows + 31) / 32 * 32;   // no group has more than there are
  args.stage_bytes = (kBOff + rows * kBK + 1023) / 1024 * 1024;
  args.stages = std::min(kMaxStages, (kSmemBytes - kFixedBytes) / args.stage_bytes);
  args.err = device_error_word();
  if (!ok || args.err == nullptr) return FP8Q_ERR_CUDA;
  return out_dtype == FP8Q_DT_BF16 ? run_split<__nv_bfloat16>(maps, args, stream)
                                   : run_split<float>(maps, args, stream);
}

}  // namespace experts
}  // namespace fp8q
