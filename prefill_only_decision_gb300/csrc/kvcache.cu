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
// sides of a warp cover whole 128-byte lines, hd / 8 threads per vector.
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"

namespace s1 {
namespace kvc {

constexpr int THREADS = 256;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<f16>(f16 x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<bf16>(bf16 x) { return __bfloat162float(x); }

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

// Eight consecutive elements; VEC: the address is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float* x) {
  T t[8];
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(t)[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f<T>(t[i]);
}
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

// grid (vectors * LPV / THREADS, 2 planes): vector i = row * Hkv + head.
template <typename T, int HD, bool VEC>
__global__ void __launch_bounds__(THREADS)
    quant_kernel(const T* k, const T* v, int64_t k_stride, int64_t v_stride, uint32_t n_vec, int Hkv, uint8_t* codes,
                 float* scales, int cap, int pos0) {
  constexpr int LPV = HD / 8;
  allow_dependents();
  wait_prerequisites();
  const uint32_t i = blockIdx.x * (THREADS / LPV) + threadIdx.x / LPV;
  const int l = threadIdx.x % LPV;
  const bool live = i < n_vec;               // (shuffles below take whole warps)
  const uint32_t row = live ? i / (uint32_t)Hkv : 0, h = live ? i % (uint32_t)Hkv : 0;
  const int plane = blockIdx.y;
  const T* src = plane ? v + (int64_t)row * v_stride : k + (int64_t)row * k_stride;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) load8<T, VEC>(src + (int64_t)h * HD + l * 8, x);
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaxf(a, isfinite(x[e]) ? fabsf(x[e]) : 0.f);
#pragma unroll
  for (int o = LPV / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (!live) return;
  const int E = scale_exp(a);
  const float inv = pow2(-E);                // -120 .. 126
  uint16_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  const int64_t crow = (int64_t)plane * cap + pos0 + row;
  *reinterpret_cast<uint2*>(codes + (crow * Hkv + h) * HD + l * 8) =
      make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
  if (l == 0) scales[((int64_t)plane * Hkv + h) * cap + pos0 + row] = pow2(E);
}

template <typename T, int HD, bool VEC>
__global__ void __launch_bounds__(THREADS)
    dequant_kernel(const uint8_t* codes, const float* scales, int cap, int pos0, uint32_t n_vec, int Hkv, T* k, T* v,
                   int64_t k_stride, int64_t v_stride) {
  constexpr int LPV = HD / 8;
  allow_dependents();
  wait_prerequisites();
  const uint32_t i = blockIdx.x * (THREADS / LPV) + threadIdx.x / LPV;
  const int l = threadIdx.x % LPV;
  if (i >= n_vec) return;
  const uint32_t row = i / (uint32_t)Hkv, h = i % (uint32_t)Hkv;
  const int plane = blockIdx.y;
  const int64_t crow = (int64_t)plane * cap + pos0 + row;
  const uint2 c = __ldcs(reinterpret_cast<const uint2*>(codes + (crow * Hkv + h) * HD + l * 8));
  const float s = scales[((int64_t)plane * Hkv + h) * cap + pos0 + row];
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? c.x : c.y;
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (e & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    x[2 * e] = f.x * s;
    x[2 * e + 1] = f.y * s;
  }
  T* dst = plane ? v + (int64_t)row * v_stride : k + (int64_t)row * k_stride;
  store8<T, VEC>(dst + (int64_t)h * HD + l * 8, x);
}

// Rows whose every vector starts on a 16-byte boundary.
inline bool rows_aligned(const void* k, const void* v, int64_t ks, int64_t vs, int esize) {
  return (((uintptr_t)k | (uintptr_t)v | (uintptr_t)(ks * esize) | (uintptr_t)(vs * esize)) & 15) == 0;
}

// Vectors of one launch: 32-bit indices, grid.x well below its limit.
constexpr int64_t MAX_VEC = 1 << 28;

}  // namespace kvc

template <typename T, int HD, bool VEC>
static cudaError_t quant_t(const T* k, const T* v, int64_t ks, int64_t vs, int rows, int Hkv, uint8_t* codes,
                           float* scales, int cap, int pos0, cudaStream_t st) {
  const int per = kvc::THREADS / (HD / 8);
  const int step = (int)std::max<int64_t>(1, kvc::MAX_VEC / Hkv);
  for (int r = 0; r < rows; r += std::min(step, rows - r)) {
    const uint32_t n_vec = (uint32_t)((int64_t)std::min(step, rows - r) * Hkv);
    CK_RET(launch_pdl(kvc::quant_kernel<T, HD, VEC>, dim3((n_vec + per - 1) / per, 2), dim3(kvc::THREADS), 0, st,
                      k + (int64_t)r * ks, v + (int64_t)r * vs, ks, vs, n_vec, Hkv, codes, scales, cap, pos0 + r));
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
    CK_RET(launch_pdl(kvc::dequant_kernel<T, HD, VEC>, dim3((n_vec + per - 1) / per, 2), dim3(kvc::THREADS), 0, st,
                      codes, scales, cap, pos0 + r, n_vec, Hkv, k + (int64_t)r * ks, v + (int64_t)r * vs, ks, vs));
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
