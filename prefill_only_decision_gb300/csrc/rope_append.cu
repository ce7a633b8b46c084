// Rotary positions of rows, and rows rotated on their way into a paged cache.
//
// Pair i of a head is turned by pos * w_i. In fp32 that angle is lost at far positions (2^20 radians: an error
// of 0.06), and fp64 is slow here; turns as integers are neither: w_i / 2 pi modulo 1 in units of 2^-64 times the position
// is one 64-bit product whose overflow is the whole turns. Its top 32 bits give the quadrant and an angle within an eighth
// of a turn, whose sine and cosine fp32 holds to its last bit or two.
//
// Every element is read and written once: HBM bound. A block takes RB rows: it computes the rows' n_pairs sines and cosines
// once into shared memory for all heads (a sine in every thread that uses one would cost five times the rotation
// itself), then a thread turns 2 x 8 elements of a head at a time, chunk c and its partner chunk, hd / 16 threads a
// head, U of them loaded before the first is used.
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kvrows.cuh"

namespace s1 {
namespace rap {
using kvc::Raw;

constexpr int THREADS = 256, RB_MAX = 4;

// cos and sin of pos * turn (2^-64 turns).
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t turn) {
  const uint64_t ph = (uint64_t)(int64_t)pos * turn;
  const uint32_t p = (uint32_t)((ph + 0x80000000ull) >> 32);
  const uint32_t quad = (p + 0x20000000u) >> 30;
  const int r = (int)(p - (quad << 30));                     // -2^29 .. 2^29 - 1
  float s, c;
  sincospif((float)r * 4.656612873077392578125e-10f, &s, &c);   // 2^-31
  const float x = quad & 1 ? s : c, y = quad & 1 ? c : s;
  return make_float2(quad == 1 || quad == 2 ? -x : x, quad >= 2 ? -y : y);
}

__device__ __forceinline__ uint32_t pack16(f16, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack16(bf16, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store8_16(T* p, const float* x, bool vec) {
  const uint4 w = make_uint4(pack16(T(), x[0], x[1]), pack16(T(), x[2], x[3]), pack16(T(), x[4], x[5]),
                             pack16(T(), x[6], x[7]));
  if (vec) {
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    T t[8];
    memcpy(t, &w, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = t[i];
  }
}
// Eight elements at element offset `off` of an array of the given ElemType.
__device__ __forceinline__ void store8(void* base, int64_t off, int type, const float* x, bool vec) {
  if (type == ELEM_F16) {
    store8_16((f16*)base + off, x, vec);
  } else if (type == ELEM_BF16) {
    store8_16((bf16*)base + off, x, vec);
  } else {
    float* p = (float*)base + off;
    if (vec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
  }
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& r, float* x) {
  T t[8];
  memcpy(t, &r, sizeof(t));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = kvc::to_f(t[i]);
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __int_as_float(0x7f800000) ? a : 0.f;           // (NaN: 0)
}

// grid (row blocks of rb rows, head blocks of hb heads): heads 0 .. Hq-1 are q's, then k's, then v's.
template <typename T, int HD, bool VEC, bool APPEND>
__global__ void __launch_bounds__(THREADS) rows_kernel(const __grid_constant__ RowsArgs a, int rb, int hb, bool out_vec) {
  constexpr int NU = HD / 16, U = sizeof(T) == 4 ? 2 : 4;
  __shared__ float4 cs[RB_MAX * MAX_PAIRS / 2];              // (cos, sin) pairs
  __shared__ int64_t place[RB_MAX];                          // of a row in a plane of pages: vector (head 0); -1: none
  __shared__ int live[RB_MAX];
  allow_dependents();
  wait_prerequisites();
  const int np = a.rope.n_pairs, np8 = np / 8;
  const int r0 = blockIdx.x * rb, rows = min(rb, a.n_rows - r0);
  const int H = a.Hq + (APPEND ? 2 * a.pages.Hkv : 0);
  const int h0 = blockIdx.y * hb, heads = min(hb, H - h0);
  for (int i = threadIdx.x; i < rows * np; i += THREADS) {
    const int row = i / np, pair = i - row * np;
    const int p = !APPEND || a.pos ? a.pos[a.rope.axis[pair] * a.pos_stride + r0 + row] : a.at[r0 + row];
    reinterpret_cast<float2*>(cs)[row * MAX_PAIRS + pair] = cos_sin(p, a.rope.turn[pair]);
  }
  if (threadIdx.x < rows) {
    const int row = r0 + threadIdx.x;
    int64_t at = -1;
    int on = 1;
    if constexpr (APPEND) {
      const int j = a.at[row], s = a.seq ? a.seq[row] : row;
      on = j >= 0;
      const int col = j >> a.pages.shift;
      if (on && s >= 0 && s < a.pages.n_seq && col < a.pages.cols) {
        const int id = a.pages.table[s * a.pages.table_stride + col];
        if (id >= 0 && id < a.pages.n_pages)
          at = (((int64_t)id * a.pages.Hkv) << a.pages.shift) + (j & ((1 << a.pages.shift) - 1));
      }
    }
    place[threadIdx.x] = at;
    live[threadIdx.x] = on;
  }
  __syncthreads();
  const int total = rows * heads * NU;
  for (int b = 0; b < total; b += THREADS * U) {             // (the whole block: lanes past the end take part in shuffles)
    Raw<T> x[U][2];
    int row[U], h[U], c0[U], c1[U];
    bool turn[U], in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = b + u * THREADS + threadIdx.x;
      in[u] = i < (uint32_t)total;
      const int unit = i % NU;
      const uint32_t hr = in[u] ? i / NU : 0;
      row[u] = hr / (uint32_t)heads;
      h[u] = h0 + hr - row[u] * heads;
      in[u] = in[u] && live[row[u]];
      const T* src = (const T*)a.q + (r0 + row[u]) * a.q_stride + (int64_t)h[u] * HD;
      bool rotated = true;
      if constexpr (APPEND) {
        if (h[u] >= a.Hq) {
          const int hk = h[u] - a.Hq;
          rotated = hk < a.pages.Hkv;
          in[u] = in[u] && place[row[u]] >= 0;
          src = rotated ? (const T*)a.k + (r0 + row[u]) * a.k_stride + (int64_t)hk * HD
                        : (const T*)a.v + (r0 + row[u]) * a.v_stride + (int64_t)(hk - a.pages.Hkv) * HD;
        }
      }
      const int n8 = rotated ? np8 : 0;
      turn[u] = unit < n8;                                   // chunks c and c + n8; past the pairs, side by side halves
      c0[u] = turn[u] ? unit : unit + n8;
      c1[u] = turn[u] ? unit + n8 : unit + NU;
      x[u][0] = x[u][1] = Raw<T>{};
      if (in[u]) {
        x[u][0] = kvc::load8<T, VEC>(src + c0[u] * 8);
        x[u][1] = kvc::load8<T, VEC>(src + c1[u] * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lo[8], hi[8];
      widen(x[u][0], lo);
      widen(x[u][1], hi);
      if (turn[u]) {
        const float4* t = cs + (row[u] * MAX_PAIRS + c0[u] * 8) / 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 w = t[e];
          const float a0 = lo[2 * e], b0 = hi[2 * e], a1 = lo[2 * e + 1], b1 = hi[2 * e + 1];
          lo[2 * e] = a0 * w.x - b0 * w.y;
          hi[2 * e] = b0 * w.x + a0 * w.y;
          lo[2 * e + 1] = a1 * w.z - b1 * w.w;
          hi[2 * e + 1] = b1 * w.z + a1 * w.w;
        }
      }
      if constexpr (APPEND) {
        float m = 0.f;
        if (a.pages.format == KVF_E4M3) {                    // the head's largest finite magnitude
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(finite_abs(lo[e]), finite_abs(hi[e])));
#pragma unroll
          for (int o = NU / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        if (!in[u]) continue;
        if (h[u] >= a.Hq) {
          const int hk = h[u] - a.Hq, plane = hk >= a.pages.Hkv, kvh = hk - plane * a.pages.Hkv;
          const int64_t vec = (((int64_t)plane * a.pages.n_pages * a.pages.Hkv + kvh) << a.pages.shift) + place[row[u]];
          if (a.pages.format == KVF_E4M3) {
            const int E = kvc::scale_exp(m);
            const float inv = kvc::pow2(-E);
            uint8_t* codes = (uint8_t*)a.pages.data + vec * HD;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float* y = half ? hi : lo;
              uint16_t c[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                c[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * e] * inv, y[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
              *reinterpret_cast<uint2*>(codes + (half ? c1[u] : c0[u]) * 8) = kvc::pack_codes(c);
            }
            if (threadIdx.x % NU == 0) a.pages.scales[vec] = kvc::pow2(E);
          } else {
            const int type = a.pages.format == KVF_F16 ? ELEM_F16 : ELEM_BF16;
            store8(a.pages.data, vec * HD + c0[u] * 8, type, lo, true);
            store8(a.pages.data, vec * HD + c1[u] * 8, type, hi, true);
          }
          continue;
        }
      }
      if (!in[u]) continue;
      const int64_t o = (r0 + row[u]) * a.q_out_stride + (int64_t)h[u] * HD;
      store8(a.q_out, o + c0[u] * 8, a.q_out_type, lo, out_vec);
      store8(a.q_out, o + c1[u] * 8, a.q_out_type, hi, out_vec);
    }
  }
}

template <typename T, int HD, bool VEC, bool APPEND>
cudaError_t launch_t(const RowsArgs& a, bool out_vec, cudaStream_t st) {
  const int H = a.Hq + (APPEND ? 2 * a.pages.Hkv : 0);
  constexpr int NU = HD / 16;
  // few rows: one row and 256 threads' worth of heads a block, so that they spread over the SMs
  const bool small = (int64_t)a.n_rows * H * NU < 2ll * 152 * 2048;
  const int rb = small ? 1 : RB_MAX, hb = small ? std::min(H, THREADS / NU) : H;
  const dim3 grid((a.n_rows + rb - 1) / rb, (H + hb - 1) / hb);
  return launch_pdl(rows_kernel<T, HD, VEC, APPEND>, grid, dim3(THREADS), 0, st, a, rb, hb, out_vec);
}
template <typename T, int HD>
cudaError_t launch_vec(const RowsArgs& a, cudaStream_t st) {
  auto ok = [](const void* p, int64_t stride, int es) { return (((uintptr_t)p | (uintptr_t)(stride * es)) & 15) == 0; };
  const bool append = a.k != nullptr;
  const int es = sizeof(T);
  const bool vec = ok(a.q, a.q_stride, es) && (!append || (ok(a.k, a.k_stride, es) && ok(a.v, a.v_stride, es)));
  const bool out_vec = ok(a.q_out, a.q_out_stride, a.q_out_type == ELEM_F32 ? 4 : 2);
  if (append) return vec ? launch_t<T, HD, true, true>(a, out_vec, st) : launch_t<T, HD, false, true>(a, out_vec, st);
  return vec ? launch_t<T, HD, true, false>(a, out_vec, st) : launch_t<T, HD, false, false>(a, out_vec, st);
}
template <typename T>
cudaError_t launch_hd(const RowsArgs& a, cudaStream_t st) {
  return a.hd == 128 ? launch_vec<T, 128>(a, st) : launch_vec<T, 64>(a, st);
}
}  // namespace rap

cudaError_t launch_rope_rows(const RowsArgs& a, int dtype, cudaStream_t st) {
  if (dtype == ELEM_F32) return rap::launch_hd<float>(a, st);
  return dtype == ELEM_F16 ? rap::launch_hd<f16>(a, st) : rap::launch_hd<bf16>(a, st);
}

}  // namespace s1
