// Eight consecutive elements of a row in their storage type, as the casting
// kernels of the 4-bit and activation-checkpoint operators hold them: bf16
// stays packed two to a register.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8q {
namespace pack8 {

// The larger magnitudes of two pairs of bf16, NaN if either is one; the signs
// of the result mean nothing.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename T>
struct Pack8;

template <>
struct Pack8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load_vec(const __nv_bfloat16 *p) {
    const uint4 t = *reinterpret_cast<const uint4 *>(p);
    w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
  }
  __device__ __forceinline__ void take(int, const uint4 &t) { w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w; }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load_some(const __nv_bfloat16 *p, int valid) {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (2 * k < valid ? (uint32_t)q[2 * k] : 0u) |
             (2 * k + 1 < valid ? (uint32_t)q[2 * k + 1] << 16 : 0u);
  }
  __device__ __forceinline__ float2 pair(int k) const {
    return make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  }
  __device__ __forceinline__ float at(int j) const {
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
  // max |element| as an fp32 bit pattern (NaN sorts above infinity)
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t m = max_abs2(max_abs2(w[0], w[1]), max_abs2(w[2], w[3])) & 0x7FFF7FFFu;
    return max(m << 16, m & 0xFFFF0000u);
  }
};

template <>
struct Pack8<float> {
  float v[8];
  __device__ __forceinline__ void load_vec(const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  // 16-byte part h of the eight elements
  __device__ __forceinline__ void take(int h, const uint4 &t) {
    v[4 * h] = __uint_as_float(t.x), v[4 * h + 1] = __uint_as_float(t.y);
    v[4 * h + 2] = __uint_as_float(t.z), v[4 * h + 3] = __uint_as_float(t.w);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ void load_some(const float *p, int valid) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? p[j] : 0.0f;
  }
  __device__ __forceinline__ float2 pair(int k) const { return make_float2(v[2 * k], v[2 * k + 1]); }
  __device__ __forceinline__ float at(int j) const { return v[j]; }
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
  }
};

// Elements [0, valid) of a row from p, zeros after; VEC: p is 16-byte aligned
// and valid is 0 or 8.
template <bool VEC, typename T>
__device__ __forceinline__ void load(Pack8<T> &x, const T *p, int valid) {
  if (!VEC) {
    x.load_some(p, valid);
  } else if (valid > 0) {
    x.load_vec(p);
  } else {
    x.clear();
  }
}

// Two values to two bf16 elements, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

template <bool STREAM, typename V>
__device__ __forceinline__ void put(V *p, V v) {
  if (STREAM)
    __stcs(p, v);
  else
    *p = v;
}

// VEC: p is 16-byte aligned and valid is 0 or 8.  STREAM: first out of L2 (a
// large result that is not read here; 2-4% of the activation kernels' time).
template <bool VEC, bool STREAM = false, typename T>
__device__ __forceinline__ void store(T *p, int valid, const float (&v)[8]) {
  if (VEC) {
    if (valid <= 0) return;
    if constexpr (sizeof(T) == 2) {
      put<STREAM>(reinterpret_cast<uint4 *>(p),
                  make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                             bf16x2(v[6], v[7])));
    } else {
      put<STREAM>(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
      put<STREAM>(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) p[j] = (T)v[j];
}

// Asynchronous copy of 16 bytes (both sides aligned) into shared memory;
// nothing is read and zeros are written where `on` is false.
__device__ __forceinline__ void copy_async16(void *dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared::cta.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(on ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's newest groups are still under way.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace pack8
}  // namespace fp8q
