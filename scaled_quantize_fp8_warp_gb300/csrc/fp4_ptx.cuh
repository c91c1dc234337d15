// Inline-PTX wrappers for the 4-bit block-scaled MMA (tcgen05.mma
// kind::mxf4nvf4), written from the public PTX ISA description.
#pragma once

#include <stdint.h>

#include "../../include/fp8q.h"
#include "fp8q_ptx.cuh"

namespace fp8q {
namespace ptx {

// Instruction descriptor for kind::mxf4nvf4, both operands E2M1 and K-major,
// K = 64 per instruction: scale-word half of B in [4,6) and of A in [29,31)
// (0 or 2: which two bytes of the 32-bit word, for one scale per 32), A / B
// formats in [7,10) / [10,12) (1 = E2M1), N >> 3 in [17,23), scale type in
// bit 23 (0 = UE4M3, 1 = UE8M0), M >> 7 in [27,29).
__host__ __device__ constexpr uint32_t idesc_fp4(int kind, uint32_t m, uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) |
         ((kind == FP4Q_MXFP4 ? 1u : 0u) << 23) | ((m >> 7) << 27);
}

// D[tmem] (+)= (A . SFA) . (B . SFB)^T over 64 K, scales read from tensor
// memory: two bytes a row for MXFP4 (one scale per 32), four for NVFP4 (one
// per 16).
template <int KIND>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                        uint32_t accumulate) {
  if (KIND == FP4Q_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// The same for a CTA pair (cta_group::2), issued by one thread of the even
// CTA: M = 256, each CTA holding 128 rows of A, half of B's rows, the scales
// of its own rows of A and those of all of B.
template <int KIND>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t sfa_tmem,
                                             uint32_t sfb_tmem, uint32_t accumulate) {
  if (KIND == FP4Q_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// tmem_cp_32x128b_x4 in both CTAs of the pair, each from its own shared
// memory at the descriptor's address into its own tensor memory.
__device__ __forceinline__ void tmem_cp_32x128b_x4_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// True in one lane of a converged warp.  tcgen05 instructions take their
// descriptors from uniform registers: code under this predicate keeps them
// there, where code under a lane comparison moves every operand of every
// instruction across (64 to 77 cycles an instruction, measured).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// A counter in shared memory that one thread raises and others wait for.
__device__ __forceinline__ void counter_set(uint32_t addr, int value) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(addr), "r"(value) : "memory");
}
__device__ __forceinline__ int counter_get(uint32_t addr) {
  int v;
  asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Bounded wait of a converged warp for a counter above `value` (as
// wait_bounded_all for a barrier).
__device__ __forceinline__ bool wait_counter_all(uint32_t addr, int value,
                                                 volatile int *abort_flag, unsigned int *err) {
  uint64_t t0 = 0;
  uint32_t spins = 0;
  while (true) {
    if (__all_sync(0xFFFFFFFFu, counter_get(addr) > value)) return true;
    if ((spins++ & 255u) == 0) {
      int verdict = 0;   // 1: another thread aborted, 2: this wait ran out of time
      if ((threadIdx.x & 31) == 0) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        verdict = *abort_flag ? 1 : (now - t0 > kWaitLimitNs ? 2 : 0);
      }
      verdict = __shfl_sync(0xFFFFFFFFu, verdict, 0);
      if (verdict != 0) {
        if (verdict == 2 && (threadIdx.x & 31) == 0) {
          *abort_flag = 1;
          atomicOr(err, 1u);
        }
        return false;
      }
    }
  }
}

// Every thread of every CTA in the cluster: release this CTA's prior writes,
// wait for all the others.  Not the .aligned form, whose warps must be
// converged: threads come here from loops of different lengths, and an arrival
// counted twice would let a CTA leave while another still reads its memory.
__device__ __forceinline__ void cluster_sync_any() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 32 bytes to global memory, streaming (written once, not read here).
__device__ __forceinline__ void store_32b(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

}  // namespace ptx
}  // namespace fp8q
