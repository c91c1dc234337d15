// The product of two 4-bit operands, C = A . B^T, on the tensor cores' own
// block scaling (tcgen05.mma kind::mxf4nvf4): every K block's scales are
// copied from shared into tensor memory (tcgen05.cp) ahead of its MMAs, the
// whole K range accumulates in fp32 in tensor memory, and the epilogue
// multiplies by the tensor scales (NVFP4), converts and stores.
//
// A ring stage holds 256 elements of K (128 bytes a row, 128-byte swizzle):
// 128 rows of A, 256 of B, and the scale atoms of both (one 512-byte atom per
// 128 rows and 128 (MXFP4) or 64 (NVFP4) of K).  Tensor memory: the
// accumulator in columns [0, 256), then one slot of scales per ring stage.
#include <cuda.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "fp4_common.cuh"
#include "fp4_internal.h"
#include "fp4_ptx.cuh"
#include "fp8q_gemm_common.cuh"

namespace fp8q {
namespace fp4 {
namespace {

using namespace ptx;

constexpr int kBM = 128, kBN = 256;
constexpr int kBKBytes = 128;          // bytes of K per stage
constexpr int kBK = 256;               // elements of K per stage
constexpr int kStages = 4;

struct Args {
  int64_t M, N;
  int num_m_tiles, num_n_tiles, num_k_blocks;
  int num_steps;            // MMAs of 64 K over all of K
  int atoms_k;              // scale atoms along K
  int group, along_n;       // raster
  uint32_t idesc;
  void *C;
  const uint8_t *sfa, *sfb;
  const float *ga, *gb;     // NVFP4 tensor scales
  unsigned int *err;
};

template <int KIND>
struct Layout {
  static constexpr int kAtoms = kBK / Kind<KIND>::kAtomK;     // per stage and 128 rows: 2 or 4
  static constexpr int kABytes = kBM * kBKBytes, kBBytes = kBN * kBKBytes;
  static constexpr int kSfaOff = kABytes + kBBytes;
  static constexpr int kSfbOff = kSfaOff + kAtoms * 512;       // B's two row blocks, one after the other
  static constexpr int kStageBytes = (kSfbOff + 2 * kAtoms * 512 + 1023) / 1024 * 1024;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kBarBytes = 8 * (2 * kStages + 3);
  static constexpr int kSmemBytes = kRingBytes + kBarBytes + 16 + 1024;
  static constexpr uint32_t kSfCol0 = kBN;
  static constexpr uint32_t kSfCols = 12 * kAtoms;             // A: 4 columns an atom, B: 8
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSfCol0 + kSfCols * kStages <= kTmemCols, "scale slots fit in TMEM");
  static_assert(kSmemBytes <= 227 * 1024, "the ring fits in shared memory");
};

// 32 consecutive results of row m from column n0.  VEC: every row of C starts
// on a 16-byte boundary, so whole groups of 16 bytes are stored at once.
template <typename T, bool VEC>
__device__ __forceinline__ void store32(T *C, int64_t N, int64_t m, int64_t n0,
                                        const float (&v)[32]) {
  constexpr int kVec = 16 / sizeof(T);
  T *row = C + m * N + n0;
#pragma unroll
  for (int g = 0; g < 32 / kVec; ++g) {
    if (VEC) {
      if (n0 + g * kVec < N) {
        __align__(16) T w[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) w[j] = (T)v[g * kVec + j];
        __stcs(reinterpret_cast<uint4 *>(row + g * kVec), *reinterpret_cast<const uint4 *>(w));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (n0 + g * kVec + j < N) row[g * kVec + j] = (T)v[g * kVec + j];
    }
  }
}

template <int KIND, typename T, bool VEC>
__global__ void __launch_bounds__(320, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const Args p) {
  using L = Layout<KIND>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + L::kRingBytes;
  const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
  const uint32_t accf = bars + 8 * (2 * kStages), acce = accf + 8, drain = acce + 8;
  const uint32_t slot = bars + L::kBarBytes;
  uint8_t *slot_ptr = smem_raw + (slot - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slot_ptr + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
    mbar_init(acce, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
  }
  if (warp == 1) {
    tmem_alloc(slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(slot_ptr);
  const int total = p.num_m_tiles * p.num_n_tiles;
  const int num_nb = (int)((p.N + 127) / 128);   // 128-row blocks of B

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        int mt, nt;
        gemm::tile_coords(u, p.num_m_tiles, p.num_n_tiles, mt, nt, p.group, p.along_n);
        const int nbv = min(2, num_nb - 2 * nt);   // B's row blocks inside the matrix
        for (int kb = 0; kb < p.num_k_blocks; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          const uint32_t full = full0 + 8 * s;
          if (!wait_bounded(empty0 + 8 * s, ph ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + s * L::kStageBytes;
          const int ka = kb * L::kAtoms;
          const uint32_t bytes = 512u * (uint32_t)min(L::kAtoms, p.atoms_k - ka);
          mbar_arrive_expect_tx(full, L::kABytes + L::kBBytes + bytes * (1u + (uint32_t)nbv));
          tma_load_2d(sa, &ta, kb * kBKBytes, mt * kBM, full);
          tma_load_2d(sa + L::kABytes, &tb, kb * kBKBytes, nt * kBN, full);
          bulk_load(sa + L::kSfaOff, p.sfa + ((int64_t)mt * p.atoms_k + ka) * 512, bytes, full);
          for (int h = 0; h < nbv; ++h)
            bulk_load(sa + L::kSfbOff + h * L::kAtoms * 512,
                      p.sfb + ((int64_t)(2 * nt + h) * p.atoms_k + ka) * 512, bytes, full);
        }
      }
      if (!ok) {
        // Let the copies already issued land before the CTA goes away.
        const uint32_t n = it < (uint32_t)kStages ? it : (uint32_t)kStages;
        for (uint32_t j = 0; j < n; ++j) {
          const uint32_t jj = it - 1 - j;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full0 + 8 * (jj % kStages), (jj / kStages) & 1u) &&
                 globaltimer_ns() - t0 < 200000000ull) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, acc_it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++acc_it) {
        if (!wait_bounded(acce, (acc_it & 1u) ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < p.num_k_blocks; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!wait_bounded(full0 + 8 * s, ph, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = ring + s * L::kStageBytes;
          const uint32_t sfa = tmem_base + L::kSfCol0 + L::kSfCols * s;
          const uint32_t sfb = sfa + 4 * L::kAtoms;
#pragma unroll
          for (int a = 0; a < L::kAtoms; ++a) {
            tmem_cp_32x128b_x4(sfa + 4 * a, sdesc_plain(sa + L::kSfaOff + 512 * a, 128));
            tmem_cp_32x128b_x4(sfb + 8 * a, sdesc_plain(sa + L::kSfbOff + 512 * a, 128));
            tmem_cp_32x128b_x4(sfb + 8 * a + 4,
                               sdesc_plain(sa + L::kSfbOff + 512 * (L::kAtoms + a), 128));
          }
          // the last block may hold fewer than four steps: K past the matrix
          // would multiply zeros with scales that were not loaded
          const int steps = min(4, p.num_steps - 4 * kb);
          for (int k = 0; k < steps; ++k) {
            const uint64_t ad = sdesc_k(sa + 32 * k, gemm::kSwzSBO, gemm::kSwzMode);
            const uint64_t bd = sdesc_k(sa + L::kABytes + 32 * k, gemm::kSwzSBO, gemm::kSwzMode);
            const int a = KIND == FP4Q_MXFP4 ? k >> 1 : k;
            const uint32_t half = KIND == FP4Q_MXFP4 ? 2u * (k & 1) : 0u;
            mma_fp4<KIND>(tmem_base, ad, bd, p.idesc | (half << 29) | (half << 4), sfa + 4 * a,
                          sfb + 8 * a, (kb > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(empty0 + 8 * s);
        }
        if (!ok) break;
        mma_commit(accf);
      }
      gemm::drain_mma(drain, abort_flag);
    }
    __syncwarp();
  } else {
    // Warps 2..9: warp w drains TMEM lane quarter w % 4, columns
    // [128 h, 128 h + 128) with h = (w - 2) / 4.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const float g = KIND == FP4Q_NVFP4 ? __fmul_rn(*p.ga, *p.gb) : 1.0f;
    uint32_t acc_it = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++acc_it) {
      int mt, nt;
      gemm::tile_coords(u, p.num_m_tiles, p.num_n_tiles, mt, nt, p.group, p.along_n);
      if (!wait_bounded_warp(accf, acc_it & 1u, abort_flag, p.err)) break;
      tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + half * 128 + c * 32,
                           r[c]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce);   // the accumulator is free for the next tile
      const int64_t m = (int64_t)mt * kBM + quarter * 32 + lane;
      if (m < p.M) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t n0 = (int64_t)nt * kBN + half * 128 + c * 32;
          if (n0 < p.N) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = KIND == FP4Q_NVFP4 ? __fmul_rn(__uint_as_float(r[c][j]), g)
                                        : __uint_as_float(r[c][j]);
            store32<T, VEC>(static_cast<T *>(p.C), p.N, m, n0, v);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, L::kTmemCols);
}

template <int KIND, typename T, bool VEC>
int run(const CUtensorMap &ta, const CUtensorMap &tb, const Args &a, cudaStream_t stream) {
  auto kernel = gemm_kernel<KIND, T, VEC>;
  static PerDeviceOnce setup;  // per instantiation
  if (setup.get([&] {
        return gemm::set_smem(kernel, Layout<KIND>::kSmemBytes) == cudaSuccess ? 1 : 0;
      }) != 1)
    return FP8Q_ERR_CUDA;
  const int64_t tiles = (int64_t)a.num_m_tiles * a.num_n_tiles;
  kernel<<<(int)std::min<int64_t>(tiles, sm_count()), 320, Layout<KIND>::kSmemBytes, stream>>>(
      ta, tb, a);
  return cudaGetLastError() == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
}

template <int KIND, typename T>
int run_vec(const CUtensorMap &ta, const CUtensorMap &tb, const Args &a, cudaStream_t stream) {
  return a.N * (int64_t)sizeof(T) % 16 == 0 ? run<KIND, T, true>(ta, tb, a, stream)
                                            : run<KIND, T, false>(ta, tb, a, stream);
}

bool make_tmap(CUtensorMap *m, const void *base, int64_t rows, int64_t K, uint32_t box_rows) {
  const uint64_t bytes = (uint64_t)row_bytes(K);
  return make_tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, bytes, (uint64_t)rows, bytes,
                      kBKBytes, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

int launch_gemm(int kind, const fp4q_operand &A, const fp4q_operand &B, int out_dtype, void *C,
                int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
  CUtensorMap ta, tb;
  if (!make_tmap(&ta, A.data, M, K, kBM) || !make_tmap(&tb, B.data, N, K, kBN))
    return FP8Q_ERR_CUDA;
  Args a{};
  a.M = M;
  a.N = N;
  a.num_m_tiles = (int)((M + kBM - 1) / kBM);
  a.num_n_tiles = (int)((N + kBN - 1) / kBN);
  a.num_k_blocks = (int)((K + kBK - 1) / kBK);
  a.num_steps = (int)((K + 63) / 64);
  a.atoms_k = (int)num_atoms_k(kind, K);
  a.group = 16;
  a.along_n = 0;
  a.idesc = idesc_fp4(kind, kBM, kBN);
  a.C = C;
  a.sfa = A.scales;
  a.sfb = B.scales;
  a.ga = A.global_scale;
  a.gb = B.global_scale;
  a.err = device_error_word();
  if (a.err == nullptr) return FP8Q_ERR_CUDA;
  if ((int64_t)a.num_m_tiles * a.num_n_tiles > INT32_MAX / 2) return FP8Q_ERR_INVALID_ARG;
  if (log_enabled())
    fprintf(stderr, "[fp8q] launch fp4 gemm_kernel %lldx%lldx%lld kind %d out %d\n", (long long)M,
            (long long)N, (long long)K, kind, out_dtype);
  if (kind == FP4Q_MXFP4)
    return out_dtype == FP8Q_DT_BF16 ? run_vec<FP4Q_MXFP4, __nv_bfloat16>(ta, tb, a, stream)
                                     : run_vec<FP4Q_MXFP4, float>(ta, tb, a, stream);
  return out_dtype == FP8Q_DT_BF16 ? run_vec<FP4Q_NVFP4, __nv_bfloat16>(ta, tb, a, stream)
                                   : run_vec<FP4Q_NVFP4, float>(ta, tb, a, stream);
}

}  // namespace fp4
}  // namespace fp8q
