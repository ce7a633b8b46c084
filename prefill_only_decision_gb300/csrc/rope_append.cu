// Rotary positions of rows, and rows rotated on their way into a paged cache.
//
// Pair i of a head is turned by pos * w_i. In fp32 that angle is lost at far positions (2^20 radians: an error of
// 0.06), and fp64 is slow here; turns as integers are neither: w_i / 2 pi modulo 1 in units of 2^-64 times the
// position is one 64-bit product whose overflow is the whole turns. Its top 32 bits (an angle is rounded to 2^-32 turns)
// give the quadrant and an angle within an eighth of a turn, whose sine and cosine are within 2^-23.
//
// Every element is read and written once: HBM bound. A block takes tiles of RB rows in turn: for each it makes the
// rows' n_pairs sines and cosines once into shared memory for all heads (a sine in every thread that uses one would
// cost five times the rotation itself), then a thread turns 2 x 8 elements of a head at a time, chunk c and its
// partner chunk, hd / 16 threads a head, U of them loaded before the first is used. Blocks stay because a thread then
// looks its pair's frequency up once (lanes that index kernel parameters differently are served one by one: 70001
// rows to e4m3 192 us with a block per tile), and so that the next tile's positions and page ids are on their way
// under the present one.
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kvrows.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace rap {
using namespace t5;
using kvc::Raw;

constexpr int THREADS = 256, RB_MAX = 16, PASSES = 4;         // rows of a tile; angles of a tile that a thread makes

// cos and sin of pos * turn (2^-64 turns): quadrant and rest, the rest's Taylor series (|y| <= pi / 4: the terms left
// out are below 2^-28 of the sine and 2^-32 of the cosine).
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t turn) {
  const uint64_t ph = (uint64_t)(int64_t)pos * turn;
  const uint32_t p = (uint32_t)((ph + 0x80000000ull) >> 32);
  const uint32_t quad = (p + 0x20000000u) >> 30;
  const float y = (float)(int)(p - (quad << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float z = y * y;
  const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), y);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float u = quad & 1 ? s : c, v = quad & 1 ? c : s;
  return make_float2(quad == 1 || quad == 2 ? -u : u, quad >= 2 ? -v : v);
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
// Two pairs (lo[i], hi[i]) turned at once.
__device__ __forceinline__ void turn2(float* lo, float* hi, uint64_t c, uint64_t s, uint64_t minus_s) {
  const uint64_t a = pack2(lo[0], lo[1]), b = pack2(hi[0], hi[1]);
  const uint64_t x = fma2(a, c, mul2(b, minus_s)), y = fma2(b, c, mul2(a, s));
  lo[0] = lo2(x);
  lo[1] = hi2(x);
  hi[0] = lo2(y);
  hi[1] = hi2(y);
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

// grid (row blocks of rb rows, head blocks of hb heads): heads 0 .. Hq-1 are q's, then k's, then v's. U, the units a
// thread loads at once: 2, and 1 where a call is small. Blocks of an SM: 4 with 16-bit rows, 3 with fp32 ones, whose
// loads take twice the registers (70001 rows f16 to e4m3 with 3, 4, 5 blocks: 157, 147, 163 us; 12345 rows f32 to
// bf16 40.6, 46, 61 us; U of 1, 3, 4 f16: 165, 152, 162 us; 37 tokens with U of 1 and 2: 2.9, 3.4 us).
constexpr int blocks_of(size_t es) { return es == 4 ? 3 : 4; }
template <typename T, int HD, bool VEC, bool APPEND, int U>
__global__ void __launch_bounds__(THREADS, blocks_of(sizeof(T)))
    rows_kernel(const __grid_constant__ RowsArgs a, int rb, int hb, bool out_vec) {
  constexpr int NU = HD / 16;
  __shared__ float4 cs[2][RB_MAX][2][MAX_PAIRS / 4];         // cosines, then sines, by tile parity and row
  __shared__ int64_t place[2][RB_MAX];                       // of a row in a plane of pages: vector (head 0); -1: none
  __shared__ int live[2][RB_MAX];
  allow_dependents();
  const int np = a.rope.n_pairs, np8 = np / 8;
  const int H = a.Hq + (APPEND ? 2 * a.pages.Hkv : 0);
  const int h0 = blockIdx.y * hb, heads = min(hb, H - h0);
  const uint32_t magic = 0xffffffffu / (uint32_t)heads + 1;
  // this thread's angles: pair tpair of rows trow, trow + rstep, .. of each tile
  const int rstep = np ? THREADS / np : 1, trow = np ? (int)threadIdx.x / np : RB_MAX;
  const int tpair = np ? (int)threadIdx.x - trow * np : 0;
  const bool angles = np && trow < min(rb, rstep);
  uint64_t turn = 0;
  int64_t axis = 0;
  if (angles) {
    const uint64_t* t = a.rope.turn;
    const uint8_t* x = a.rope.axis;
    asm volatile("" : "+l"(t), "+l"(x));                     // (loads, not indexed constants)
    turn = t[tpair];
    axis = x[tpair];
  }
  wait_prerequisites();
  const int tiles = (a.n_rows + rb - 1) / rb;
  int pos[PASSES];                                           // a tile ahead of their use
  auto positions = [&](int tile) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int rr = trow + i * rstep;
      pos[i] = 0;
      if (!angles || tile >= tiles || rr >= rb || tile * rb + rr >= a.n_rows) continue;
      pos[i] = !APPEND || a.pos ? a.pos[axis * a.pos_stride + tile * rb + rr] : a.at[tile * rb + rr];
    }
  };
  // threads 0 .. rb - 1: where the tile's rows go
  struct Where {
    int j, s;
  };
  auto where = [&](int tile) {
    Where w = {-1, 0};
    const int r = tile * rb + (int)threadIdx.x;
    if (!APPEND || threadIdx.x >= rb || tile >= tiles || r >= a.n_rows) return w;
    w.j = a.at[r];
    w.s = a.seq ? a.seq[r] : r;
    return w;
  };
  auto page_of = [&](const Where& w) {                       // -1: none
    if (!APPEND || w.j < 0 || w.s < 0 || w.s >= a.pages.n_seq || w.j >> a.pages.shift >= a.pages.cols) return -1;
    const int id = a.pages.table[w.s * a.pages.table_stride + (w.j >> a.pages.shift)];
    return id < a.pages.n_pages ? id : -1;
  };
  int r0, total;                                             // of the tile at hand: first row, units
  Raw<T> x[U][2];
  int row[U], h[U];
  // unit i: rows' heads in turn, hd / 16 units a head; two chunks c0 and c1 of 8 elements: a pair's two sides, or
  // past the pairs two that stay
  auto chunk0 = [&](int unit, int n8) { return unit < n8 ? unit : unit + n8; };
  auto chunk1 = [&](int unit, int n8) { return unit < n8 ? unit + n8 : unit + NU; };
  const int unit = threadIdx.x % NU;                         // (THREADS is a multiple of NU)
  auto pairs8 = [&](int head) { return !APPEND || head < a.Hq + a.pages.Hkv ? np8 : 0; };
  auto load = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * THREADS + (int)threadIdx.x;
      const int hr = i / NU;
      const int r = heads == 1 ? hr : (int)__umulhi((uint32_t)hr, magic);   // hr / heads (hr < 16 heads, heads < 2^14)
      row[u] = i < total ? r : -1;
      h[u] = h0 + hr - r * heads;
      x[u][0] = x[u][1] = Raw<T>{};
      if (row[u] < 0) continue;
      const T* src = (const T*)a.q + (r0 + r) * a.q_stride + (int64_t)h[u] * HD;
      if constexpr (APPEND)
        if (h[u] >= a.Hq) {
          const int hk = h[u] - a.Hq;
          src = hk < a.pages.Hkv ? (const T*)a.k + (r0 + r) * a.k_stride + (int64_t)hk * HD
                                 : (const T*)a.v + (r0 + r) * a.v_stride + (int64_t)(hk - a.pages.Hkv) * HD;
        }
      const int n8 = pairs8(h[u]);
      x[u][0] = kvc::load8<T, VEC>(src + chunk0(unit, n8) * 8);
      x[u][1] = kvc::load8<T, VEC>(src + chunk1(unit, n8) * 8);
    }
  };
  positions(blockIdx.x);
  Where w = where(blockIdx.x), w_next = where(blockIdx.x + gridDim.x);
  int id = page_of(w);
  for (int tile = blockIdx.x, buf = 0; tile < tiles; tile += gridDim.x, buf ^= 1) {
    r0 = tile * rb;
    total = min(rb, a.n_rows - r0) * heads * NU;
    load(0);                                                   // (in flight while the angles are made)
    if (angles)
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
        if (trow + i * rstep < rb) {
          const float2 t = cos_sin(pos[i], turn);
          float* at = reinterpret_cast<float*>(cs[buf][trow + i * rstep]) + tpair;
          at[0] = t.x;
          at[MAX_PAIRS] = t.y;
        }
    if (APPEND && threadIdx.x < rb) {
      const int64_t first = ((int64_t)id * a.pages.Hkv) << a.pages.shift;
      place[buf][threadIdx.x] = id < 0 ? -1 : first + (w.j & ((1 << a.pages.shift) - 1));
      live[buf][threadIdx.x] = w.j >= 0;
    }
    __syncthreads();                                         // (one a tile: the other buffer's readers passed the one before)
    positions(tile + gridDim.x);
    w = w_next;
    id = page_of(w);
    w_next = where(tile + 2 * gridDim.x);
    for (int b = 0; b < total; b += THREADS * U) {             // (the whole block: lanes past the end take part in shuffles)
      if (b) load(b);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float lo[8], hi[8];
        widen(x[u][0], lo);
        widen(x[u][1], hi);
        const int n8 = pairs8(h[u]), c0 = chunk0(unit, n8), c1 = chunk1(unit, n8), r = max(row[u], 0);
        if (unit < n8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 c = cs[buf][r][0][c0 * 2 + e], s = cs[buf][r][1][c0 * 2 + e];
            turn2(lo + 4 * e, hi + 4 * e, pack2(c.x, c.y), pack2(s.x, s.y), pack2(-s.x, -s.y));
            turn2(lo + 4 * e + 2, hi + 4 * e + 2, pack2(c.z, c.w), pack2(s.z, s.w), pack2(-s.z, -s.w));
          }
        }
        bool in = row[u] >= 0;
        if constexpr (APPEND) {
          float m = 0.f;
          if (a.pages.format == KVF_E4M3 && __any_sync(0xffffffffu, in && h[u] >= a.Hq)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(lo[e]), fabsf(hi[e])));   // (NaN: left out)
            if (isinf(m)) {                                    // the head's largest finite magnitude
              m = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(finite_abs(lo[e]), finite_abs(hi[e])));
            }
#pragma unroll
            for (int o = NU / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          }
          in = in && live[buf][r];
          if (in && h[u] >= a.Hq) {
            if (place[buf][r] < 0) continue;
            const int hk = h[u] - a.Hq, plane = hk >= a.pages.Hkv, kvh = hk - plane * a.pages.Hkv;
            const int64_t vec = (((int64_t)plane * a.pages.n_pages * a.pages.Hkv + kvh) << a.pages.shift) + place[buf][r];
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
                *reinterpret_cast<uint2*>(codes + (half ? c1 : c0) * 8) = kvc::pack_codes(c);
              }
              if (unit == 0) a.pages.scales[vec] = kvc::pow2(E);
            } else {
              const int type = a.pages.format == KVF_F16 ? ELEM_F16 : ELEM_BF16;
              store8(a.pages.data, vec * HD + c0 * 8, type, lo, true);
              store8(a.pages.data, vec * HD + c1 * 8, type, hi, true);
            }
            continue;
          }
        }
        if (!in) continue;
        const int64_t o = (r0 + r) * a.q_out_stride + (int64_t)h[u] * HD;
        store8(a.q_out, o + c0 * 8, a.q_out_type, lo, out_vec);
        store8(a.q_out, o + c1 * 8, a.q_out_type, hi, out_vec);
      }
    }
  }
}

template <typename T, int HD, bool VEC, bool APPEND>
cudaError_t launch_t(const RowsArgs& a, bool out_vec, int num_sms, cudaStream_t st) {
  const int H = a.Hq + (APPEND ? 2 * a.pages.Hkv : 0);
  constexpr int NU = HD / 16;
  // A tile holds enough rows for one or two of a thread's batches; fewer where the rows then would not reach all SMs,
  // and of few rows a block takes the heads of one batch of loads. At most 8192 heads a block.
  const int want = std::max(PASSES, (4 * THREADS + H * NU - 1) / (H * NU));
  int rb = 1;
  // (1280 rows f16 with at least one, two, four tiles an SM: 7.4, 6.9, 6.1 us; 1500 rows f32 9.6, 6.9, 7.8)
  const int enough = (sizeof(T) == 4 ? 2 : 4) * num_sms;
  while (rb < RB_MAX && rb < want && a.n_rows >= 2 * rb * enough) rb *= 2;
  rb = std::min(rb, PASSES * (a.rope.n_pairs ? THREADS / a.rope.n_pairs : THREADS));
  const int hb = rb >= 4 ? std::min(H, 8192) : std::min(H, THREADS / NU);
  const dim3 grid(std::min((a.n_rows + rb - 1) / rb, blocks_of(sizeof(T)) * num_sms), (H + hb - 1) / hb);
  return launch_pdl(rb >= 4 ? rows_kernel<T, HD, VEC, APPEND, 2> : rows_kernel<T, HD, VEC, APPEND, 1>, grid, dim3(THREADS),
                    0, st, a, rb, hb, out_vec);
}
template <typename T, int HD>
cudaError_t launch_vec(const RowsArgs& a, int num_sms, cudaStream_t st) {
  auto ok = [](const void* p, int64_t stride, int es) { return (((uintptr_t)p | (uintptr_t)(stride * es)) & 15) == 0; };
  const bool append = a.k != nullptr;
  const int es = sizeof(T);
  const bool vec = ok(a.q, a.q_stride, es) && (!append || (ok(a.k, a.k_stride, es) && ok(a.v, a.v_stride, es)));
  const bool out_vec = ok(a.q_out, a.q_out_stride, a.q_out_type == ELEM_F32 ? 4 : 2);
  if (append)
    return vec ? launch_t<T, HD, true, true>(a, out_vec, num_sms, st) : launch_t<T, HD, false, true>(a, out_vec, num_sms, st);
  return vec ? launch_t<T, HD, true, false>(a, out_vec, num_sms, st) : launch_t<T, HD, false, false>(a, out_vec, num_sms, st);
}
template <typename T>
cudaError_t launch_hd(const RowsArgs& a, int num_sms, cudaStream_t st) {
  return a.hd == 128 ? launch_vec<T, 128>(a, num_sms, st) : launch_vec<T, 64>(a, num_sms, st);
}
}  // namespace rap

cudaError_t launch_rope_rows(const RowsArgs& a, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == ELEM_F32) return rap::launch_hd<float>(a, num_sms, st);
  return dtype == ELEM_F16 ? rap::launch_hd<f16>(a, num_sms, st) : rap::launch_hd<bf16>(a, num_sms, st);
}

}  // namespace s1
