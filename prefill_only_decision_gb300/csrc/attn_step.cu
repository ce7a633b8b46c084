// Attention of one new token of each sequence over a paged cache: o = softmax(scale q.K^T) V over the rows that the
// token sees, every cached row read once for the (up to 16) q heads that share its kv head.
//
// Bound by HBM: 4 hd flops per q head for 4 hd bytes of an f16 row (K and V), 5 q heads: 5 flops a byte. So the split is
// made for the memory system: the work of a call is the list of all 64-row tiles of all (sequence, kv head) pairs, and
// CTA c of C (one per SM) takes the c-th of C equal runs of it, whatever the sequences' lengths. The runs follow from pos,
// which every CTA reads on the device (a captured call stays balanced as positions grow). A run covers some pairs wholly,
// which are written at once, and at most two in part, whose (o, m, l) join_kernel joins in the order of the CTAs: the
// sizes and positions fix every order of summation.
//
// A CTA: warp 8 asks for the tiles by TMA (a lane per page box; page ids read 32 columns ahead) into a ring that holds
// some 190 KB; 8 warps compute, four on the even and four on the odd tiles, 16 rows each, without any exchange until the pair
// ends. With at most 16 query rows tcgen05's 128-row tiles would stand nearly empty and pass S and P through TMEM between
// warps, so the products are mma.sync's m16n8k16, whose operands and results stay in one warp's registers: Q as the A operand, scores
// in the layout in which P is the next A operand. Each warp keeps a running base and sum of its own rows.
//
// e4m3 pages: the codes travel and are widened to f16 in registers. The sums over d and over rows do not care for
// their order, so both products take the codes in the order in which wide shared-memory reads find them: key column
// n of a product stands for row key8(n), and thread (g, t) holds chunk t of a K row (16 d's as four k-steps) and chunk g
// of V rows (16 columns of the product's tiles). K scales multiply the scores. V scales go into the weights as exponents: the
// base is a running bound of z + e (V's scale 2^e f, f in [1/2, 1)), so neither f16 nor the sums see the scales' range.
// bf16 queries over e4m3 pages become f16 by a power of two per row.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "paged.cuh"

namespace s1 {
namespace pgs {
using namespace t5;
using namespace pga;

constexpr int KT = 64, WARPS = 8, THREADS = (WARPS + 1) * 32;
enum Kind { F16 = 0, BF16 = 1, E4M3 = 2 };

__device__ uint64_t g_given_up;              // when a bounded wait last gave up, per device; never cleared

template <int HD, int KIND>
struct Lay {
  static constexpr int PLANE = KT * HD * (KIND == E4M3 ? 1 : 2), TILE = 2 * PLANE;
  static constexpr int NST = KIND == E4M3 ? (HD == 128 ? 10 : 16) : (HD == 128 ? 6 : 12);   // even
  static constexpr int SC = NST * TILE;                       // scales of a stage: [2][KT] floats (e4m3)
  static constexpr int OSTR = HD + 4;                         // floats of a row in a warp's published sums
  static constexpr int OUT = SC + (KIND == E4M3 ? NST * 2 * KT * 4 : 0);
  static constexpr int ML = OUT + WARPS * 8 * OSTR * 4;       // [WARPS][8] (m, l)
  static constexpr int BAR = ML + WARPS * 8 * 8;
  static constexpr int BYTES = BAR + 2 * NST * 8 + 64;
  static_assert(BYTES + 1024 <= 227 * 1024 && NST % 2 == 0, "shared memory of one CTA");
};

struct StepArgs {
  PagedAttnArgs a;
  const int* pos;
  int n, G, HG, groups;      // q heads per kv head; (kv head, group of 16 q heads) pairs of a sequence, groups per kv head
};

// Part slots of the workspace: slot 2 c for the pair that CTA c's run continues, 2 c + 1 for the one that it starts and does not
// end; 16 rows of hd sums, then 16 (m, l). Behind them a record for each CTA: the pair whose last tile its run holds.
struct Record {
  int seq, hg, first, valid;   // first: the CTA with the pair's first tile
};
__host__ __device__ constexpr int64_t slot_floats(int hd) { return 16 * (hd + 2); }

// Where score column n (0 .. 7) of a product's key tile lies among its 8 rows.
template <int KIND>
__device__ __forceinline__ int key8(int n) {
  return KIND == E4M3 ? (n & 1 ? (n ^ 4) : n) : n;
}
// The column of O that element e (0, 1) of thread t's accumulator of tile b stands for.
template <int HD, int KIND>
__device__ __forceinline__ int out_col(int b, int t, int e) {
  return KIND == E4M3 ? (HD / 8) * (2 * t + e) + b : 8 * b + 2 * t + e;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {   // two e4m3 codes (low 16 bits) to an f16 pair
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return (uint32_t)r.y << 16 | r.x;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack_w(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return h2u(a, b);
  }
}
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // the 8 computing warps

// A run's position in the list of tiles.
struct Cursor {
  int s, hg, t, T;
  Seen v;
  Tiles tl;
};

template <int HD, int KIND, bool QBF>
__global__ void __launch_bounds__(THREADS, 1)
    step_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ StepArgs sa) {
  using L = Lay<HD, KIND>;
  constexpr int NST = L::NST;
  constexpr bool PBF = KIND == BF16;           // the products' type
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = (uint64_t*)(sm + L::BAR);   // [NST]
  uint64_t* empty = full + NST;                // [NST]
  volatile int* abort_flag = (volatile int*)(empty + NST);
  int* found = (int*)(empty + NST) + 1;        // the run's first sequence
  __shared__ int64_t red[WARPS + 1];
  __shared__ int64_t found_before;             // tiles (per pair) of the sequences before it
  const PagedAttnArgs& a = sa.a;
  const PagesArgs& pg = a.pages;
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  allow_dependents();
  wait_prerequisites();

  // ---- this CTA's run of the list of tiles
  const int rows = (int)(((int64_t)pg.cols) << pg.shift);
  auto look = [&](Cursor& c, int s) {
    c.s = s;
    c.v = seen_rows(sa.pos[s], rows, a.window, a.sinks);
    c.tl = tiles_of<KT>(c.v);
    c.T = c.tl.count();
  };
  auto tiles_at = [&](int s) { return s < sa.n ? tiles_of<KT>(seen_rows(sa.pos[s], rows, a.window, a.sinks)).count() : 0; };
  auto block_scan = [&](int64_t x, int64_t* total) {          // inclusive, over the block's threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w <= WARPS; ++w) {
      if (w < warp) before += red[w];
      all += red[w];
    }
    *total = all;
    return x + before;
  };
  int64_t per_head = 0, first_scan = 0;
  for (int b = 0; b < sa.n; b += THREADS) {
    int64_t t;
    const int64_t x = block_scan(tiles_at(b + (int)threadIdx.x), &t);
    if (b == 0) first_scan = x;
    per_head += t;
  }
  const int64_t units = per_head * sa.HG;
  const int64_t C = min(units, (int64_t)gridDim.x);          // CTAs with a run: none of them is empty
  const int64_t u0 = blockIdx.x < C ? units * blockIdx.x / C : 0, u1 = blockIdx.x < C ? units * (blockIdx.x + 1) / C : 0;
  if (u0 < u1) {                               // the first sequence whose tiles reach beyond u0
    int64_t carry = 0;
    bool there = false;
    for (int b = 0; b < sa.n && !there; b += THREADS) {
      int64_t t;
      const int s = b + (int)threadIdx.x;
      const int64_t mine = tiles_at(s), x = b == 0 ? first_scan : block_scan(mine, &t);
      if (b == 0) t = INT64_MAX;
      const int64_t end = carry + x;
      if (end * sa.HG > u0 && (end - mine) * sa.HG <= u0) {
        *found = s;
        found_before = end - mine;
      }
      __syncthreads();
      if (b == 0) {                            // (the first block's total again: the last thread's)
        if (threadIdx.x == THREADS - 1) red[0] = x;
        __syncthreads();
        t = red[0];
      }
      carry += t;
      there = carry * sa.HG > u0;
    }
  }
  __syncthreads();
  Cursor c0 = {};
  if (u0 < u1) {
    look(c0, *found);
    const int64_t r = u0 - found_before * sa.HG;
    c0.hg = (int)(r / c0.T);
    c0.t = (int)(r % c0.T);
  }
  // runs fn(cursor, tiles of the pair in this run) over the pairs of the run
  auto each_pair = [&](auto&& fn) {
    Cursor c = c0;
    for (int64_t u = u0; u < u1;) {
      const int m = (int)min((int64_t)(c.T - c.t), u1 - u);
      if (!fn(c, m)) return;
      u += m;
      c.t = 0;
      if (u < u1 && ++c.hg == sa.HG) {
        c.hg = 0;
        do look(c, c.s + 1);
        while (c.T == 0);
      }
    }
  };

  int asked = 0;                               // tiles asked for (producer)
  if (warp == WARPS) {
    // ---- TMA producer
    constexpr int NB = KIND == E4M3 ? 1 : HD / 64;
    const int npg = pg.shift < 6 ? KT >> pg.shift : 1, br = KT / npg;     // pages of a tile, rows of a box
    const int plane = lane & 1, box = (lane >> 1) % NB, part = (lane >> 1) / NB;
    int& i = asked;
    each_pair([&](const Cursor& c, int m) {
      const int64_t trow = (int64_t)c.s * pg.table_stride;
      const int head = c.hg / sa.groups, last = (c.v.end - 1) >> pg.shift;
      int blk = -1, cur = 0, next = 0;         // page ids of columns 32 blk .. +31, and of the block behind them
      auto ids = [&](int b) {
        const int col = b * 32 + lane;
        return col <= last ? pg.table[trow + col] : -1;
      };
      for (int t = c.t; t < c.t + m; ++t, ++i) {
        const int j0 = c.tl.at(t) * KT, col = j0 >> pg.shift;
        if (col >> 5 != blk) {
          cur = blk >= 0 && col >> 5 == blk + 1 ? next : ids(col >> 5);
          blk = col >> 5;
          next = ids(blk + 1);
        }
        const int id = __shfl_sync(0xffffffffu, cur, (col + part) & 31);
        const int st = i % NST;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], (i / NST & 1) ^ 1, abort_flag, &g_given_up) ? 1 : 0)) return false;
        uint8_t* dst = sm + st * L::TILE;
        const int there = min(npg, last - col + 1);            // pages that the sequence has
        const bool valid = id >= 0 && id < pg.n_pages;
        uint32_t bytes = (uint32_t)(there * br) * (HD * (KIND == E4M3 ? 1 : 2) * 2);
        if constexpr (KIND == E4M3) {
          // scales: 64 to 256 contiguous bytes of a page; of a page that does not exist, ones
          float* sc = (float*)(sm + L::SC) + st * 2 * KT + plane * KT + part * br;
          const bool mine = lane < npg * 2 && part < there;
          const uint32_t n_valid = __popc(__ballot_sync(0xffffffffu, mine && valid));
          bytes += n_valid * (uint32_t)br * 4;
          if (mine && !valid) {
            for (int r = 0; r < br; ++r) sc[r] = 1.f;
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&full[st], bytes);
          __syncwarp();
          if (mine && valid)
            bulk_load(sc, pg.scales + ((((int64_t)plane * pg.n_pages + id) * pg.Hkv + head) << pg.shift) +
                              (j0 & ((1 << pg.shift) - 1)), br * 4, &full[st]);
        } else {
          if (lane == 0) mbar_expect_tx(&full[st], bytes);
          __syncwarp();
        }
        if (lane < npg * NB * 2 && part < there)
          tma5(dst + plane * L::PLANE + box * (KT * 128) + part * br * (KIND == E4M3 ? HD : 128), &map, &full[st], box * 64,
               j0 & ((1 << pg.shift) - 1), head, id, plane);
      }
      return true;
    });
  } else {
    // ---- computing warps: rows 16 sub .. +15 of every second tile
    const int grp = warp >> 2, sub = warp & 3, g = lane >> 2, t4 = lane & 3;
    const float sl2 = a.scale * 1.4426950408889634f;
    float* pub = (float*)(sm + L::OUT);
    float2* ml = (float2*)(sm + L::ML);
    const uint32_t base_k = smem_u32(sm);
    bool ok = true;
    int i = 0;                                 // tiles of the run before the pair
    // tokens that see nothing: zeros
    for (int s = blockIdx.x; s < sa.n; s += gridDim.x)
      if (sa.pos[s] < 0 || tiles_at(s) == 0)
        for (int e = threadIdx.x; e < a.Hq * HD / 8; e += WARPS * 32)
          reinterpret_cast<uint4*>((uint16_t*)a.out + (int64_t)s * a.Hq * HD)[e] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
      Record* rec = reinterpret_cast<Record*>((float*)a.ws + 2 * (int64_t)gridDim.x * slot_floats(HD)) + blockIdx.x;
      rec->valid = 0;
    }
    each_pair([&](const Cursor& c, int m) {
      const int kvh = c.hg / sa.groups, h0 = kvh * sa.G + (c.hg % sa.groups) * 16;
      const int nq = min(16, (kvh + 1) * sa.G - h0);           // q heads of the pair
      // Q as A fragments: rows g and g + 8; d of k-step ks as the K operand has it
      uint32_t q[HD / 16][4];
      float qs0 = sl2, qs1 = sl2;                              // what a score of row g, g + 8 is multiplied by
      {
        const uint16_t* qp = (const uint16_t*)a.q + (int64_t)c.s * a.q_stride + (int64_t)h0 * HD;
        auto row = [&](int r, int ks, int half) -> uint32_t {
          const int d = KIND == E4M3 ? 64 * (ks >> 2) + 16 * t4 + 4 * (ks & 3) + 2 * half : 16 * ks + 2 * t4 + 8 * half;
          return r < nq ? __ldg(reinterpret_cast<const uint32_t*>(qp + r * HD + d)) : 0u;
        };
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) q[ks][e] = row(g + 8 * (e & 1), ks, e >> 1);
        if constexpr (KIND == E4M3 && QBF) {                   // to f16, the row's largest element near 2^14
          uint32_t top[2] = {0, 0};
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top[e & 1] = max(top[e & 1], max(q[ks][e] & 0x7fffu, q[ks][e] >> 16 & 0x7fffu));
          float up[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = max(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = max(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            const int E = min(max((int)(top[r] >> 7) - 127, -100), 127);
            up[r] = __uint_as_float((uint32_t)(14 - E + 127) << 23);
            (r ? qs1 : qs0) *= __uint_as_float((uint32_t)(E - 14 + 127) << 23);
          }
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              q[ks][e] = h2u(__uint_as_float(q[ks][e] << 16) * up[e & 1],
                             __uint_as_float(q[ks][e] & 0xffff0000u) * up[e & 1]);
        }
      }
      float o[HD / 8][4] = {};
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      for (int x = (i + grp) & 1; x < m && ok; x += 2) {
        const int tile = i + x, st = tile % NST;
        const int j0 = c.tl.at(c.t + x) * KT + sub * 16;       // this warp's first row
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], tile / NST & 1, abort_flag, &g_given_up) ? 1 : 0)) {
          ok = false;
          break;
        }
        const bool whole = j0 + 15 < c.v.end && (j0 >= c.v.lo || j0 + 15 < c.v.sk);
        const bool none = j0 >= c.v.end || (j0 + 15 < c.v.lo && j0 >= c.v.sk);
        if (!none) {
          const uint32_t kb = base_k + st * L::TILE, vb = kb + L::PLANE;
          float s[2][4] = {};
          // ---- S = Q K^T
          if constexpr (KIND != E4M3) {
            const int r = sub * 16 + (lane & 7) + (lane & 16 ? 8 : 0), ch = lane >> 3 & 1;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
              uint32_t b[4];
              ldsm4<false>(b, kb + (ks >> 2) * (KT * 128) + r * 128 + ((((ks & 3) * 2 + ch) ^ (r & 7)) << 4));
              mma16816<PBF>(s[0], q[ks], b[0], b[1]);
              mma16816<PBF>(s[1], q[ks], b[2], b[3]);
            }
          } else {
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
              const int r = sub * 16 + nb * 8 + key8<KIND>(g);
#pragma unroll
              for (int j = 0; j < HD / 64; ++j) {
                const int ch = HD == 128 ? (4 * j + t4) ^ (r & 7) : t4 ^ (r >> 1 & 3);
                uint32_t w[4];
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(kb + r * HD + (ch << 4)));
#pragma unroll
                for (int k = 0; k < 4; ++k) mma16816<false>(s[nb], q[4 * j + k], widen2(w[k]), widen2(w[k] >> 16));
              }
            }
          }
          // ---- scores in the log2 domain, hidden rows -inf; t: what the base is taken from
          float f[2][2];                                       // e4m3: V scales' fractions by (nb, e)
          float ex[2][2];                                      // and exponents
          uint32_t hid = 0;                                    // bit 2 nb + e: the row is hidden
          if (!whole) {
#pragma unroll
            for (int x4 = 0; x4 < 4; ++x4) {
              const int j = j0 + (x4 >> 1) * 8 + key8<KIND>(2 * t4 + (x4 & 1));
              if (j >= c.v.end || (j < c.v.lo && j >= c.v.sk)) hid |= 1u << x4;
            }
          }
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float f0 = qs0, f1 = qs1;
              const bool h = hid >> (2 * nb + e) & 1;
              if constexpr (KIND == E4M3) {
                const float* sc = (const float*)(sm + L::SC) + st * 2 * KT + sub * 16 + nb * 8 + key8<KIND>(2 * t4 + e);
                f0 *= sc[0];
                f1 *= sc[0];
                const uint32_t u = __float_as_uint(sc[KT]);
                const int E = (int)(u >> 23) - 126;             // (scales below 2^-81: the rest stays in f)
                ex[nb][e] = (float)max(E, -80);
                f[nb][e] = E >= -80 ? __uint_as_float((u & 0x7fffffu) | 126u << 23) : sc[KT] * 1.208925819614629e24f;
              }
              s[nb][e] = h ? -INFINITY : s[nb][e] * f0;
              s[nb][2 + e] = h ? -INFINITY : s[nb][2 + e] * f1;
            }
          auto key = [&](int nb, int e) {                      // score, or score and exponent
            if constexpr (KIND == E4M3) return s[nb][e] + ex[nb][e & 1];
            else return s[nb][e];
          };
          float x0 = fmaxf(fmaxf(key(0, 0), key(0, 1)), fmaxf(key(1, 0), key(1, 1)));
          float x1 = fmaxf(fmaxf(key(0, 2), key(0, 3)), fmaxf(key(1, 2), key(1, 3)));
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
          const bool up0 = x0 - m0 > TOP, up1 = x1 - m1 > TOP;
          if (__any_sync(0xffffffffu, up0 || up1)) {
            const float n0 = up0 ? (fabsf(x0) < FAR ? x0 - HEAD : x0) : m0, n1 = up1 ? (fabsf(x1) < FAR ? x1 - HEAD : x1) : m1;
            const float a0 = m0 == n0 || m0 == -INFINITY ? 1.f : ex2(m0 - n0);
            const float a1 = m1 == n1 || m1 == -INFINITY ? 1.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int b = 0; b < HD / 8; ++b) {
              o[b][0] *= a0;
              o[b][1] *= a0;
              o[b][2] *= a1;
              o[b][3] *= a1;
            }
          }
          const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
          uint32_t p[4];
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float b = e < 2 ? b0 : b1;
              const float d = ex2(s[nb][e] - b);               // (e4m3: the sum's weight)
              w[e] = d;
              if constexpr (KIND == E4M3) w[e] = hid >> (2 * nb + (e & 1)) & 1 ? 0.f : ex2(s[nb][e] + ex[nb][e & 1] - b) * f[nb][e & 1];
              (e < 2 ? l0 : l1) += d;
            }
            p[2 * nb] = pack_w<PBF>(w[0], w[1]);
            p[2 * nb + 1] = pack_w<PBF>(w[2], w[3]);
          }
          // ---- O += P V; the V rows of hidden keys are zeros (0 x NaN is not)
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;   // of the pairs (2t, 2t + 1), (2t + 8, 2t + 9)
          if (!whole) {
            keep0 = (hid & 1 ? 0u : 0xffffu) | (hid & 2 ? 0u : 0xffff0000u);
            keep1 = (hid & 4 ? 0u : 0xffffu) | (hid & 8 ? 0u : 0xffff0000u);
          }
          if constexpr (KIND != E4M3) {
            const int r = sub * 16 + (lane & 15), ch = lane >> 4;
#pragma unroll
            for (int b = 0; b < HD / 8; b += 2) {
              uint32_t v[4];
              ldsm4<true>(v, vb + (b >> 3) * (KT * 128) + r * 128 + ((((b & 7) + ch) ^ (r & 7)) << 4));
              if (!whole) {
                v[0] &= keep0;
                v[1] &= keep1;
                v[2] &= keep0;
                v[3] &= keep1;
              }
              mma16816<PBF>(o[b], p, v[0], v[1]);
              mma16816<PBF>(o[b + 1], p, v[2], v[3]);
            }
          } else {
            constexpr int NW = HD / 32;                        // 32-bit words of a thread's V chunk
            uint32_t w[4][NW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = sub * 16 + (k >> 1) * 8 + key8<KIND>(2 * t4 + (k & 1));
              if constexpr (HD == 128)
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[k][0]), "=r"(w[k][1]), "=r"(w[k][NW - 2]), "=r"(w[k][NW - 1])
                             : "r"(vb + r * HD + ((g ^ (r & 7)) << 4)));
              else
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                             : "=r"(w[k][0]), "=r"(w[k][1])
                             : "r"(vb + r * HD + (((g >> 1) ^ (r >> 1 & 3)) << 4) + (g & 1) * 8));
            }
#pragma unroll
            for (int x4 = 0; x4 < NW; ++x4)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t y0 = __byte_perm(w[0][x4], w[1][x4], half ? 0x7362 : 0x5140);
                const uint32_t y1 = __byte_perm(w[2][x4], w[3][x4], half ? 0x7362 : 0x5140);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t v0 = widen2(y0 >> (16 * e)) & keep0, v1 = widen2(y1 >> (16 * e)) & keep1;
                  mma16816<false>(o[4 * x4 + 2 * half + e], p, v0, v1);
                }
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      i += m;
      // ---- the pair ends here: the warps' sums through shared memory, 8 rows at a time
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      const bool starts = c.t == 0, ends = c.t + m == c.T;
      float* slot = (float*)a.ws + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * slot_floats(HD);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (8 * half >= nq) break;
        if (t4 == 0) ml[warp * 8 + g] = half ? make_float2(m1, l1) : make_float2(m0, l0);
#pragma unroll
        for (int b = 0; b < HD / 8; ++b) {
          float* at = pub + (warp * 8 + g) * L::OSTR;
          at[out_col<HD, KIND>(b, t4, 0)] = o[b][2 * half];
          at[out_col<HD, KIND>(b, t4, 1)] = o[b][2 * half + 1];
        }
        group_sync();
        constexpr int CV = HD / 4;                             // float4 columns
        for (int e = threadIdx.x; e < 8 * CV; e += WARPS * 32) {
          const int r = e / CV, cv = e % CV;
          if (8 * half + r >= nq) continue;
          float M = -INFINITY, lsum = 0.f;
          float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w * 8 + r].x);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const float2 z = ml[w * 8 + r];
            if (z.x == -INFINITY && z.y == 0.f) continue;      // (no row, or all scores -inf)
            const float wt = z.x == M ? 1.f : ex2(z.x - M);
            const float4 v = *reinterpret_cast<const float4*>(pub + (w * 8 + r) * L::OSTR + cv * 4);
            lsum += wt * z.y;
            y.x += wt * v.x;
            y.y += wt * v.y;
            y.z += wt * v.z;
            y.w += wt * v.w;
          }
          if (starts && ends) {
            const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
            *reinterpret_cast<uint2*>((uint16_t*)a.out + ((int64_t)c.s * a.Hq + h0 + 8 * half + r) * HD + cv * 4) =
                make_uint2(pack_w<QBF>(y.x * inv, y.y * inv), pack_w<QBF>(y.z * inv, y.w * inv));
          } else {
            *reinterpret_cast<float4*>(slot + (8 * half + r) * HD + cv * 4) = y;
            if (cv == 0) reinterpret_cast<float2*>(slot + 16 * HD)[8 * half + r] = make_float2(M, lsum);
          }
        }
        group_sync();
      }
      if (ends && !starts && threadIdx.x == 0) {
        // the pair's first tile: list position u0 - c.t when this is the run's first pair (the only one it does not start)
        const int64_t at = u0 - c.t;
        int64_t f = at * C / units;                            // the CTA whose run holds it
        while (units * (f + 1) / C <= at) ++f;
        while (units * f / C > at) --f;
        Record* rec = reinterpret_cast<Record*>((float*)a.ws + 2 * (int64_t)gridDim.x * slot_floats(HD)) + blockIdx.x;
        *rec = Record{c.s, c.hg, (int)f, 1};
      }
      return true;
    });
  }
  __syncthreads();
  if (warp == WARPS && *abort_flag)            // nothing in flight when the CTA leaves
    for (int st = 0; st < NST && st < asked; ++st) mbar_drain(&full[st], (asked - 1 - st) / NST & 1);
}

// Joins the parts of the pair that CTA blockIdx.x of the step ended: slot 2 first + 1, then slots 2 c of the CTAs behind it.
// Block y takes rows y, y + gridDim.y, ...; its warps take the parts in turn, and their sums are joined in order.
constexpr int JWARPS = 8;
template <int HD, bool QBF>
__global__ void __launch_bounds__(JWARPS * 32) join_kernel(const __grid_constant__ StepArgs sa, int C) {
  __shared__ float4 py[JWARPS][32];
  __shared__ float2 pml[JWARPS];
  allow_dependents();
  wait_prerequisites();
  const float* ws = (const float*)sa.a.ws;
  const Record rec = reinterpret_cast<const Record*>(ws + 2 * (int64_t)C * slot_floats(HD))[blockIdx.x];
  if (!rec.valid) return;
  const int kvh = rec.hg / sa.groups, h0 = kvh * sa.G + (rec.hg % sa.groups) * 16, nq = min(16, (kvh + 1) * sa.G - h0);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, parts = (int)blockIdx.x - rec.first + 1;
  for (int r = blockIdx.y; r < nq; r += gridDim.y) {
    float M = -INFINITY, l = 0.f;
    float4 y = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int p = w; p < parts; p += JWARPS) {
      const float* slot = ws + (p == 0 ? 2 * (int64_t)rec.first + 1 : 2 * (int64_t)(rec.first + p)) * slot_floats(HD);
      const float2 z = __ldcg(reinterpret_cast<const float2*>(slot + 16 * HD) + r);
      const float4 v = lane < HD / 4 ? __ldcg(reinterpret_cast<const float4*>(slot + r * HD) + lane) : make_float4(0, 0, 0, 0);
      if (z.x == -INFINITY && z.y == 0.f) continue;
      const float N = fmaxf(M, z.x), a0 = M == N || l == 0.f ? 1.f : ex2(M - N), a1 = z.x == N ? 1.f : ex2(z.x - N);
      M = N;
      l = a0 * l + a1 * z.y;
      y = make_float4(a0 * y.x + a1 * v.x, a0 * y.y + a1 * v.y, a0 * y.z + a1 * v.z, a0 * y.w + a1 * v.w);
    }
    py[w][lane] = y;
    if (lane == 0) pml[w] = make_float2(M, l);
    __syncthreads();
    if (w == 0 && lane < HD / 4) {
      float N = -INFINITY, s = 0.f;
      float4 o = make_float4(0, 0, 0, 0);
      for (int k = 0; k < JWARPS; ++k) N = fmaxf(N, pml[k].x);
      for (int k = 0; k < JWARPS; ++k) {
        const float2 z = pml[k];
        if (z.x == -INFINITY && z.y == 0.f) continue;
        const float wt = z.x == N ? 1.f : ex2(z.x - N);
        const float4 v = py[k][lane];
        s += wt * z.y;
        o = make_float4(o.x + wt * v.x, o.y + wt * v.y, o.z + wt * v.z, o.w + wt * v.w);
      }
      const float inv = s == 0.f ? 0.f : 1.f / s;
      *reinterpret_cast<uint2*>((uint16_t*)sa.a.out + ((int64_t)rec.seq * sa.a.Hq + h0 + r) * HD + lane * 4) =
          make_uint2(pack_w<QBF>(o.x * inv, o.y * inv), pack_w<QBF>(o.z * inv, o.w * inv));
    }
    __syncthreads();
  }
}

template <int HD, int KIND, bool QBF>
cudaError_t launch(const StepArgs& sa, int num_sms, cudaStream_t st) {
  using L = Lay<HD, KIND>;
  CUtensorMap map;
  if (!pages_map(&map, sa.a.pages, std::min(KT, 1 << sa.a.pages.shift))) return cudaErrorInvalidValue;
  CK_RET(cudaFuncSetAttribute(step_kernel<HD, KIND, QBF>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  CK_RET(launch_pdl(step_kernel<HD, KIND, QBF>, dim3((unsigned)num_sms), dim3(THREADS), L::BYTES, st, map, sa));
  return launch_pdl(join_kernel<HD, QBF>, dim3((unsigned)num_sms, 4), dim3(JWARPS * 32), 0, st, sa, num_sms);
}
template <int HD>
cudaError_t launch_kind(const StepArgs& sa, int num_sms, cudaStream_t st) {
  if (sa.a.pages.format == KVF_F16) return launch<HD, F16, false>(sa, num_sms, st);
  if (sa.a.pages.format == KVF_BF16) return launch<HD, BF16, true>(sa, num_sms, st);
  return sa.a.bf16 ? launch<HD, E4M3, true>(sa, num_sms, st) : launch<HD, E4M3, false>(sa, num_sms, st);
}
}  // namespace pgs

cudaError_t attention_step_gave_up_word(uint64_t** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), pgs::g_given_up);
}

int64_t attention_paged_step_ws_bytes(int, int, int, int hd, int num_sms) {
  return (int64_t)num_sms * (2 * pgs::slot_floats(hd) * 4 + (int64_t)sizeof(pgs::Record));
}

cudaError_t launch_attention_paged_step(const PagedAttnArgs& a, int n, const int* pos, int num_sms, cudaStream_t st) {
  pgs::StepArgs sa{a, pos, n, a.Hq / a.pages.Hkv, 0, 0};
  sa.groups = (sa.G + 15) / 16;
  sa.HG = sa.groups * a.pages.Hkv;
  return a.pages.hd == 128 ? pgs::launch_kind<128>(sa, num_sms, st) : pgs::launch_kind<64>(sa, num_sms, st);
}

}  // namespace s1
