// What the attention kernels over a paged cache share: which rows a query sees, and page tiles by TMA.
#pragma once
#include "common.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace pga {

// Weights are 2^(z - m), z the score (log2 domain) and m a base that a row moves to HEAD below its maximum when they
// would pass 2^TOP, within f16: a weight keeps f16's precision down to 2^-24 of the largest (a base at the maximum
// would lose what lies behind a sink). Maxima past FAR are their own base: fp32 does not hold HEAD beside them.
constexpr float HEAD = 10.f, TOP = 15.f, FAR = 4194304.f;

// The rows that a query at position p sees: [0, sk) and [lo, end).
struct Seen {
  int end, lo, sk;
};
__host__ __device__ __forceinline__ Seen seen_rows(int p, int rows, int window, int sinks) {
  Seen s;
  s.end = (p < rows - 1 ? p : rows - 1) + 1;
  if (s.end < 0) s.end = 0;
  s.lo = window && p - (window - 1) > 0 ? p - (window - 1) : 0;
  s.sk = sinks < s.lo ? sinks : s.lo;
  if (s.sk > s.end) s.sk = s.end;
  if (p < 0) s.end = s.lo = s.sk = 0;
  return s;
}

// Two-part tile lists: tiles [0, head) and [first, first + tail) of KT rows.
struct Tiles {
  int head, first, tail;
  __host__ __device__ int count() const { return head + tail; }
  __host__ __device__ int at(int t) const { return t < head ? t : first + t - head; }
};
template <int KT>
__host__ __device__ __forceinline__ Tiles tiles_of(const Seen& s) {
  Tiles t;
  t.first = s.lo / KT;
  t.tail = s.lo < s.end ? (s.end - 1) / KT - t.first + 1 : 0;
  t.head = (s.sk + KT - 1) / KT;
  if (t.tail && t.head > t.first) t.head = t.first;   // (the tile that both parts reach is taken once)
  return t;
}

__device__ __forceinline__ void tma5(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w,
                                     int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(t5::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(t5::smem_u32(bar))
      : "memory");
}
// 16 bytes into shared memory, zeros where !on; and an arrival (counted in the barrier's number) once this thread's
// copies are there.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(t5::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(t5::smem_u32(bar)) : "memory");
}

// Two fp32 values, rounded, as a pair of bf16 or f16.
template <bool BF>
__device__ __forceinline__ uint32_t pack_w(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return t5::h2u(a, b);
  }
}
// Four e4m3 codes to two f16 pairs.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// 2^e, e at most 127.
__device__ __forceinline__ float pow2f(int e) {
  return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : e >= -149 ? 1u << (e + 149) : 0u);
}

// Sums over e4m3 pages pass between warps, CTAs and kernels as means (o / l), since V's scales may leave fp32 no room
// beside the weights. Their l is brought to 1 .. 2 by its base (leveled), and a mean's share is l times SHARE: the
// shares of 8192 parts together are at most 1, so that no sum passes the largest mean.
constexpr float SHARE = 6.103515625e-5f, UNSHARE = 16384.f;   // 2^-14, 2^14
__device__ __forceinline__ float2 leveled(float m, float l) {
  const uint32_t u = __float_as_uint(l);
  if (!(fabsf(m) < FAR) || u - 0x800000u >= 0x7f000000u) return make_float2(m, l);   // (bases that hold no more bits; 0, NaN)
  return make_float2(m + (float)((int)(u >> 23) - 127), __uint_as_float((u & 0x7fffffu) | 127u << 23));
}

// The pages as a tensor (hd, page rows, heads, pages, planes) in boxes of `rows` rows of up to 128 bytes. A page id
// outside 0 .. n_pages - 1 is outside the tensor, which TMA reads as zeros.
inline bool pages_map(CUtensorMap* map, const PagesArgs& p, int rows) {
  const bool e4m3 = p.format == KVF_E4M3;
  const uint64_t es = e4m3 ? 1 : 2, row = p.hd * es, head = row << p.shift, page = head * p.Hkv;
  const uint64_t dims[5] = {(uint64_t)p.hd, 1ull << p.shift, (uint64_t)p.Hkv, (uint64_t)p.n_pages, 2};
  const uint64_t str[4] = {row, head, page, page * p.n_pages};
  const uint32_t box[5] = {(uint32_t)(e4m3 ? p.hd : 64), (uint32_t)rows, 1, 1, 1};
  const CUtensorMapDataType type = e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : p.format == KVF_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode_tensor_map(map, type, 5, p.data, dims, str, box,
                           e4m3 && p.hd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace pga
}  // namespace s1
