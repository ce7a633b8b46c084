// Pieces of a K/V row that the kernels which write cached rows share: eight elements as they are in memory,
// and the scale of an e4m3 vector.
#pragma once
#include <string.h>

#include "common.cuh"

namespace s1 {
namespace kvc {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(f16 x) { return __half2float(x); }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// Eight consecutive elements of a vector, as they are in memory; VEC: the address is 16-byte aligned.
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  } else {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[i];
    memcpy(&r, t, sizeof(t));
  }
  return r;
}
// The exponent E of a vector's scale from its largest finite magnitude: a = m 2^x with
// 1 <= m < 2 and 448 = 1.75 * 2^8, so E = x - 8 for m <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exp(float a) {
  if (a == 0.f) return 0;
  const uint32_t u = __float_as_uint(a);
  const int x = (int)(u >> 23) - 127;        // (subnormal a: -127, and E ends at -126)
  const int E = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return E < -126 ? -126 : E;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 .. 127

__device__ __forceinline__ uint2 pack_codes(const uint16_t* c) {
  return make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
}

}  // namespace kvc
}  // namespace s1
