// Whose turn an accumulator of the experts' products on CTA pairs is.  Tile j of
// a pair takes accumulator j % ACC for its turn j / ACC; phase t of the
// accumulator's barrier ends when every epilogue warp of both CTAs has read the
// results of turn t.  Plain arithmetic, so that the protocol can be run on a CPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FP8Q_ANYWHERE __host__ __device__ __forceinline__
#else
#define FP8Q_ANYWHERE inline
#endif

namespace fp8q {
namespace experts {

template <int ACC>
FP8Q_ANYWHERE uint32_t accumulator_of(uint32_t j) { return j % ACC; }
template <int ACC>
FP8Q_ANYWHERE uint32_t turn_of(uint32_t j) { return j / ACC; }

// Behind `tiles` tiles: wait(a, turn) for the last turn of every accumulator that
// had one, which nothing else waits for; false once a wait is.  The turn before
// it was waited for when its tile was issued, so the parity names one phase.
template <int ACC, typename Wait>
FP8Q_ANYWHERE bool settle(uint32_t tiles, Wait &&wait) {
  for (uint32_t a = 0; a < (uint32_t)ACC && a < tiles; ++a)
    if (!wait(a, turn_of<ACC>(tiles - 1 - a))) return false;
  return true;
}

}  // namespace experts
}  // namespace fp8q
