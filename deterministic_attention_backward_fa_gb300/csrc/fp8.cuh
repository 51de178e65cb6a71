// What the kernels of the 8-bit cache share (cache8.cu, decode8.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cache8.h"

namespace dash {
namespace dev {

// 2^(e - 127) of an exponent field 1 <= e <= 254
__device__ __forceinline__ float pow2_field(int e) { return __uint_as_float((uint32_t)e << 23); }

// Two e4m3 codes as two f16 of the same values.
__device__ __forceinline__ uint32_t widen8(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t narrow8(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ int quotient(const Divisor &d, int n) {
  return (int)((__umulhi((unsigned)n, d.mul) + (unsigned)n) >> d.shift);
}
template <class T>
__device__ __forceinline__ const T *wide_add(const T *p, int a, int b) {
  return p + (long long)a * b;
}
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_if(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? kBytes : 0;  // 0: fills with zeros, reads nothing
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(kBytes) : "memory");
}

}  // namespace dev
}  // namespace dash
