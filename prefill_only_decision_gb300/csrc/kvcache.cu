// The 8-bit K/V snapshot: rows quantised as they are written, and read back.
//
// Per (plane, row, head) vector x of hd elements: a = max |x| over the finite elements,
// scale = 2^E with E = ceil(log2(a / 448)) (at least -126; 0 for a = 0), code = e4m3(x / scale).
// A power of two makes the division exact, so the only rounding is e4m3's own (half a step of
// 3 mantissa bits, relative 2^-4), and the product on the way back is exact in fp32; a scale of
// a / 448 would add a rounding without a gain, since e4m3's relative step does not depend on
// where in its range a value lies.
//
// Both directions move every byte once and compute next to nothing: HBM bound. Eight elements a
// thread: a 16-byte load of f16 or bf16 (two of fp32) and an 8-byte store of codes, so that both
// sides of a warp cover whole 128-byte lines, hd / 8 threads per vector. Large calls give a thread
// U = 4 vectors, all loaded before the first is used: with one (8 bytes of codes in flight a thread
// when reading back) 150001 x 8 x 64 to bf16 ran at 4.8 TB/s (97 us) and 100000 x 8 x 128 from f16 at
// 4.3 TB/s (145 us); with four 6.2 (76 us) and 6.2 (100 us), and 100003 x 4 x 128 from fp32 at 6.7 (77
// us). Small calls keep one, and four times the blocks: 1024 rows x 4 x 128 are read back in 2.1 us.
#include <algorithm>

#include <cuda_fp8.h>

#include <string.h>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace kvc {

constexpr int THREADS = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(f16 x) { return __half2float(x); }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// x rounded to T, held at its largest finite value (NaN passes through)
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return isinf(x) ? copysignf(3.402823466e38f, x) : x;
}
template <>
__device__ __forceinline__ f16 from_f<f16>(float x) {
  return __float2half_rn(fabsf(x) > 65504.f ? copysignf(65504.f, x) : x);
}
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) {
  return __float2bfloat16_rn(fabsf(x) > 3.3895313892515355e38f ? copysignf(3.3895313892515355e38f, x) : x);
}

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
// max |x| over the finite elements. The common case (all finite) is a maximum of bit patterns, two
// 16-bit ones at a time; instructions, not bytes, bound the 16-bit types otherwise.
template <typename T>
__device__ __forceinline__ float max_finite(const Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, r.w[i] & 0x7fffffffu);
    if (m >= 0x7f800000u) {
      m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = r.w[i] & 0x7fffffffu;
        m = max(m, a < 0x7f800000u ? a : 0u);
      }
    }
    return __uint_as_float(m);
  } else {
    constexpr uint32_t TOP = std::is_same<T, f16>::value ? 0x7c00u : 0x7f80u;
    uint32_t m = t5::absmax2(T(), t5::absmax2(T(), r.w[0], r.w[1]), t5::absmax2(T(), r.w[2], r.w[3]));
    m = max(m & 0xffffu, m >> 16);
    if (m >= TOP) {
      m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = r.w[i] & 0x7fffu, hi = r.w[i] >> 16 & 0x7fffu;
        m = max(m, max(lo < TOP ? lo : 0u, hi < TOP ? hi : 0u));
      }
    }
    if constexpr (std::is_same<T, f16>::value) return __half2float(__ushort_as_half((unsigned short)m));
    else return __uint_as_float(m << 16);
  }
}
// The eight codes of x * 2^-E.
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw<T>& r, int E);

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float* x) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = from_f<T>(x[i]);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(t)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = t[i];
  }
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
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw<T>& r, int E) {
  uint16_t c[4];
  // f16: the product is exact wherever a code is not zero (a code's half step 2^-10 is a normal f16),
  // so the codes come from f16 pairs; 2^-E is an f16 number for E from -15 to 14
  if constexpr (std::is_same<T, f16>::value) {
    if (E >= -15 && E <= 14) {
      const __half2 s = __float2half2_rn(pow2(-E));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&r.w[e]), s);
        c[e] = __nv_cvt_halfraw2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      }
      return pack_codes(c);
    }
  }
  T t[8];
  memcpy(t, &r, sizeof(t));
  const float inv = pow2(-E);                // 2^-120 .. 2^126
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c[e] = __nv_cvt_float2_to_fp8x2(make_float2(to_f(t[2 * e]) * inv, to_f(t[2 * e + 1]) * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return pack_codes(c);
}

// Rows and heads of vectors i0, i0 + PER, ...: one division.
template <int PER, int U>
__device__ __forceinline__ void vectors(uint32_t i0, uint32_t Hkv, uint32_t* row, uint32_t* h) {
  row[0] = i0 / Hkv;
  h[0] = i0 - row[0] * Hkv;
  if constexpr (U > 1) {
    const uint32_t dr = PER / Hkv, dh = PER - dr * Hkv;
#pragma unroll
    for (int u = 1; u < U; ++u) {
      const uint32_t x = h[u - 1] + dh;
      const bool wrap = x >= Hkv;
      h[u] = wrap ? x - Hkv : x;
      row[u] = row[u - 1] + dr + (wrap ? 1u : 0u);
    }
  }
}

// grid (vectors * LPV / THREADS / U, 2 planes): vector i = row * Hkv + head.
template <typename T, int HD, bool VEC, int U>
__global__ void __launch_bounds__(THREADS)
    quant_kernel(const T* k, const T* v, int64_t k_stride, int64_t v_stride, uint32_t n_vec, int Hkv, uint8_t* codes,
                 float* scales, int cap, int pos0) {
  constexpr int LPV = HD / 8, PER = THREADS / LPV;
  allow_dependents();
  wait_prerequisites();
  const int l = threadIdx.x % LPV, plane = blockIdx.y;
  const uint32_t i0 = blockIdx.x * (PER * U) + threadIdx.x / LPV;
  uint32_t row[U], h[U];
  vectors<PER, U>(i0, (uint32_t)Hkv, row, h);
  Raw<T> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {              // (threads past the end take part in the shuffles with zeros)
    x[u] = Raw<T>{};
    const T* src = plane ? v + (int64_t)row[u] * v_stride : k + (int64_t)row[u] * k_stride;
    if (i0 + u * PER < n_vec) x[u] = load8<T, VEC>(src + h[u] * HD + l * 8);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float a = max_finite(x[u]);
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (i0 + u * PER >= n_vec) continue;
    const int E = scale_exp(a);
    const int64_t crow = (int64_t)plane * cap + pos0 + row[u];
    *reinterpret_cast<uint2*>(codes + (crow * Hkv + h[u]) * HD + l * 8) = codes8(x[u], E);
    if (l == 0) scales[((int64_t)plane * Hkv + h[u]) * cap + pos0 + row[u]] = pow2(E);
  }
}

template <typename T, int HD, bool VEC, int U>
__global__ void __launch_bounds__(THREADS)
    dequant_kernel(const uint8_t* codes, const float* scales, int cap, int pos0, uint32_t n_vec, int Hkv, T* k, T* v,
                   int64_t k_stride, int64_t v_stride) {
  constexpr int LPV = HD / 8, PER = THREADS / LPV;
  allow_dependents();
  wait_prerequisites();
  const int l = threadIdx.x % LPV, plane = blockIdx.y;
  const uint32_t i0 = blockIdx.x * (PER * U) + threadIdx.x / LPV;
  uint32_t row[U], h[U];
  vectors<PER, U>(i0, (uint32_t)Hkv, row, h);
  uint2 c[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (i0 + u * PER >= n_vec) continue;
    const int64_t crow = (int64_t)plane * cap + pos0 + row[u];
    c[u] = __ldcs(reinterpret_cast<const uint2*>(codes + (crow * Hkv + h[u]) * HD + l * 8));
    s[u] = scales[((int64_t)plane * Hkv + h[u]) * cap + pos0 + row[u]];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (i0 + u * PER >= n_vec) continue;
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = e < 2 ? c[u].x : c[u].y;
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (e & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      x[2 * e] = f.x * s[u];
      x[2 * e + 1] = f.y * s[u];
    }
    T* dst = plane ? v + (int64_t)row[u] * v_stride : k + (int64_t)row[u] * k_stride;
    store8<T, VEC>(dst + h[u] * HD + l * 8, x);
  }
}

// Rows whose every vector starts on a 16-byte boundary.
inline bool rows_aligned(const void* k, const void* v, int64_t ks, int64_t vs, int esize) {
  return (((uintptr_t)k | (uintptr_t)v | (uintptr_t)(ks * esize) | (uintptr_t)(vs * esize)) & 15) == 0;
}

// Vectors of one launch: 32-bit indices, grid.x well below its limit.
constexpr int64_t MAX_VEC = 1 << 28;
// Threads from which a call is large: about twice what the GPU holds at once.
constexpr int64_t LARGE = 2ll * 152 * 2048;

}  // namespace kvc

template <typename T, int HD, bool VEC>
static cudaError_t quant_t(const T* k, const T* v, int64_t ks, int64_t vs, int rows, int Hkv, uint8_t* codes,
                           float* scales, int cap, int pos0, cudaStream_t st) {
  const int per = kvc::THREADS / (HD / 8);
  const int step = (int)std::max<int64_t>(1, kvc::MAX_VEC / Hkv);
  for (int r = 0; r < rows; r += std::min(step, rows - r)) {
    const uint32_t n_vec = (uint32_t)((int64_t)std::min(step, rows - r) * Hkv);
    const bool large = 2ll * n_vec * (HD / 8) >= kvc::LARGE;
    const uint32_t bl = large ? 4 * per : per;
    CK_RET(launch_pdl(large ? kvc::quant_kernel<T, HD, VEC, 4> : kvc::quant_kernel<T, HD, VEC, 1>,
                      dim3((n_vec + bl - 1) / bl, 2), dim3(kvc::THREADS), 0, st, k + (int64_t)r * ks,
                      v + (int64_t)r * vs, ks, vs, n_vec, Hkv, codes, scales, cap, pos0 + r));
  }
  return cudaSuccess;
}
template <typename T, int HD, bool VEC>
static cudaError_t dequant_t(const uint8_t* codes, const float* scales, int cap, int pos0, int rows, int Hkv, T* k,
                             T* v, int64_t ks, int64_t vs, cudaStream_t st) {
  const int per = kvc::THREADS / (HD / 8);
  const int step = (int)std::max<int64_t>(1, kvc::MAX_VEC / Hkv);
  for (int r = 0; r < rows; r += std::min(step, rows - r)) {
    const uint32_t n_vec = (uint32_t)((int64_t)std::min(step, rows - r) * Hkv);
    const bool large = 2ll * n_vec * (HD / 8) >= kvc::LARGE;
    const uint32_t bl = large ? 4 * per : per;
    CK_RET(launch_pdl(large ? kvc::dequant_kernel<T, HD, VEC, 4> : kvc::dequant_kernel<T, HD, VEC, 1>,
                      dim3((n_vec + bl - 1) / bl, 2), dim3(kvc::THREADS), 0, st, codes, scales, cap, pos0 + r, n_vec,
                      Hkv, k + (int64_t)r * ks, v + (int64_t)r * vs, ks, vs));
  }
  return cudaSuccess;
}

// CALL(T, HD, VEC) for the runtime choice of the three.
#define KVC_DISPATCH(CALL)                                                                            \
  do {                                                                                                \
    const int es_ = dtype == ELEM_F32 ? 4 : 2;                                                        \
    const bool vec_ = kvc::rows_aligned(k, v, k_stride, v_stride, es_);                               \
    if (dtype == ELEM_F32) KVC_HD(CALL, float);                                                       \
    if (dtype == ELEM_F16) KVC_HD(CALL, f16);                                                         \
    KVC_HD(CALL, bf16);                                                                               \
  } while (0)
#define KVC_HD(CALL, T)                                                                               \
  do {                                                                                                \
    if (hd == 128) return vec_ ? CALL(T, 128, true) : CALL(T, 128, false);                            \
    return vec_ ? CALL(T, 64, true) : CALL(T, 64, false);                                             \
  } while (0)

cudaError_t launch_kv_quant(const void* k, const void* v, int dtype, int64_t k_stride, int64_t v_stride, int rows,
                            int Hkv, int hd, uint8_t* codes, float* scales, int cap, int pos0, cudaStream_t st) {
#define KVC_Q(T, HD, VEC)                                                                                            \
  quant_t<T, HD, VEC>((const T*)k, (const T*)v, k_stride, v_stride, rows, Hkv, codes, scales, cap, pos0, st)
  KVC_DISPATCH(KVC_Q);
#undef KVC_Q
}

cudaError_t launch_kv_dequant(const uint8_t* codes, const float* scales, int cap, int pos0, int rows, int Hkv, int hd,
                              void* k, void* v, int dtype, int64_t k_stride, int64_t v_stride, cudaStream_t st) {
#define KVC_D(T, HD, VEC)                                                                                            \
  dequant_t<T, HD, VEC>(codes, scales, cap, pos0, rows, Hkv, (T*)k, (T*)v, k_stride, v_stride, st)
  KVC_DISPATCH(KVC_D);
#undef KVC_D
}

}  // namespace s1
