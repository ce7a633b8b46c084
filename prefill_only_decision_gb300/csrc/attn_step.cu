// Attention of one new token of each sequence over a paged cache: o = softmax(scale q.K^T) V over the rows that the
// token sees, every cached row read once for the (up to 16) q heads that share its kv head.
//
// Bound by HBM: 4 hd flops per q head for 4 hd bytes of an f16 row (K and V), 5 q heads: 5 flops a byte. So the split
// is made for the memory system: the work of a call is the list of all 64-row tiles of all (sequence, kv head) pairs,
// and CTA c of C (one per SM) takes the c-th of C equal runs of it, whatever the sequences' lengths. The runs follow
// from pos, which every CTA reads on the device (a captured call stays balanced as positions grow). A run covers some
// pairs wholly, which are written at once, and at most two in part, whose (o, m, l) join_kernel joins in the order of
// the CTAs: the sizes and positions fix every order of summation.
//
// A CTA: three warps ask for the tiles by TMA (a lane per page box; page ids read 32 columns ahead) into a ring of
// 130 to 190 KB; the others compute, four a tile, 16 rows each, without any exchange until the pair ends. With at
// most 16 query rows tcgen05's 128-row tiles would stand nearly empty and pass S and P through TMEM between warps, so
// the products are mma.sync's m16n8k16, whose operands and results stay in one warp's registers, transposed: S^T = K
// Q^T and O^T = V^T P^T, cached rows and value columns on the 16 side and 8 q heads on the 8 side (NH = 1, or 2 for
// more than 8 heads: twice the products on the same K and V operands). One movmatrix turns 8 x 8 weights of S^T's
// layout into P^T's. Each warp keeps a running base and sum of its own rows.
//
// e4m3 pages: the codes travel and are widened to f16 in registers. The sums over d and over rows do not care for
// their order, so both products take the codes in the order in which wide shared-memory reads find them: row n of an
// 8-row block of S^T stands for cached row key8(n), and thread (g, t) holds chunk t of a K row (16 d's as four
// k-steps) and chunk g of V rows (16 columns). K scales multiply the scores. V scales go into the weights as
// exponents (V's scale 2^(unit + e) f, f in [1/2, 1), unit a warp's first; rows of scale 0, of pages that are not
// there, have no part in it): the products' base is a running bound of z + e, the sum's one of z alone, so neither f16
// nor the sums see the scales' range. bf16 queries over e4m3 pages become f16 by a power of two per q head.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "paged.cuh"

namespace s1 {
namespace pgs {
using namespace t5;
using namespace pga;

constexpr int KT = 64, PRODUCERS = 3;
constexpr int NO_UNIT = 10000;               // (e4m3) no scale yet: far above all, so that rows without one weigh nothing
constexpr int NEAR = 24;                     // (e4m3) exponents of V's scales this near the unit are ordinary
constexpr float NO_BASE = -3.402823466e38f;  // below all scores; a first one always moves it (-inf - it: no weight)
constexpr int LANE_SEQS = 8;                 // up to 32 times as many sequences are counted by each warp alone
enum Kind { F16 = 0, BF16 = 1, E4M3 = 2 };

__device__ uint64_t g_given_up;              // when a bounded wait last gave up, per device; never cleared

// Computing warps: 8, or 12 with e4m3 pages of up to 8 q heads, where widening the codes takes most of the time (16
// would leave 96 registers a thread, too few).
template <int HD, int KIND, int NH>
struct Lay {
  static constexpr int WARPS = KIND == E4M3 && NH == 1 ? 12 : 8, GROUPS = WARPS / 4;
  static constexpr int THREADS = (WARPS + PRODUCERS) * 32;
  static constexpr int PLANE = KT * HD * (KIND == E4M3 ? 1 : 2), TILE = 2 * PLANE;
  static constexpr int NST = KIND == E4M3 && NH == 1 ? (HD == 128 ? 9 : 15) : HD == 128 ? 6 : 12;
  static constexpr int SC = NST * TILE;                       // scales of a stage: [2][KT] floats (e4m3)
  static constexpr int OSTR = HD + 4;                         // floats of a q head in a warp's published sums
  static constexpr int OUT = SC + (KIND == E4M3 ? NST * 2 * KT * 4 : 0);
  static constexpr int ML = OUT + WARPS * 8 * OSTR * 4;       // [WARPS][8] (m, l)
  static constexpr int BAR = ML + WARPS * 8 * 8;
  static constexpr int BYTES = BAR + 2 * NST * 8 + 64;
  static_assert(BYTES + 1024 <= 227 * 1024, "shared memory of one CTA");
  static_assert(NST % GROUPS == 0 && NST % PRODUCERS == 0, "a stage is always the same warps' to fill and to read");
};

struct StepArgs {
  PagedAttnArgs a;
  const int* pos;
  int n, G, HG, groups;      // q heads per kv head; (kv head, group of 16 q heads) pairs of a sequence, groups per kv head
};

// Part slots of the workspace: slot 2 c for the pair that CTA c's run continues, 2 c + 1 for the one that it starts
// and does not end; 16 q heads of hd sums (means with e4m3 pages), then 16 (m, l). Behind them a record for each CTA:
// the pair whose last tile its run holds.
struct Record {
  int seq, hg, first, valid;   // first: the CTA with the pair's first tile
};
__host__ __device__ constexpr int64_t slot_floats(int hd) { return 16 * (hd + 2); }

// Where row n (0 .. 7) of an 8-row block of S^T lies among its cached rows.
template <int KIND>
__device__ __forceinline__ int key8(int n) {
  return KIND == E4M3 ? (n & 1 ? (n ^ 4) : n) : n;
}
// The value column that row g (half 0) or g + 8 (half 1) of block b of O^T stands for.
template <int HD, int KIND>
__device__ __forceinline__ int out_col(int b, int g, int half) {
  return KIND == E4M3 ? (HD / 8) * g + 2 * b + half : 16 * b + g + 8 * half;
}
// An 8 x 8 matrix of 16-bit elements, transposed over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// The computing warps.
template <int N>
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

// A run's position in the list of tiles.
struct Cursor {
  int s, hg, t, T;
  Seen v;
  Tiles tl;
};

template <int HD, int KIND, bool QBF, int NH>
__global__ void __launch_bounds__(Lay<HD, KIND, NH>::THREADS, 1)
    step_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ StepArgs sa) {
  using L = Lay<HD, KIND, NH>;
  constexpr int NST = L::NST, WARPS = L::WARPS, THREADS = L::THREADS, GROUPS = L::GROUPS;
  constexpr bool PBF = KIND == BF16;           // the products' type
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = (uint64_t*)(sm + L::BAR);   // [NST]
  uint64_t* empty = full + NST;                // [NST]
  volatile int* abort_flag = (volatile int*)(empty + NST);
  __shared__ int red[WARPS + PRODUCERS], found[2];
  const PagedAttnArgs& a = sa.a;
  const PagesArgs& pg = a.pages;
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], KIND == E4M3 ? 33 : 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  allow_dependents();
  wait_prerequisites();

  // ---- this CTA's run of the list of tiles
  const int rows = (int)(((int64_t)pg.cols) << pg.shift), HG = sa.HG;
  auto look_at = [&](Cursor& c, int s, int p) {
    c.s = s;
    c.v = seen_rows(p, rows, a.window, a.sinks);
    c.tl = tiles_of<KT>(c.v);
    c.T = c.tl.count();
  };
  auto pos_of = [&](int s) { return s < sa.n ? sa.pos[s] : -1; };
  auto tiles_at = [&](int p) { return tiles_of<KT>(seen_rows(p, rows, a.window, a.sinks)).count(); };
  auto warp_scan = [&](int x) {                // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  // the run, from the number of tiles per (kv head, group) of all sequences: the first units % C CTAs have one more
  struct Run {
    int u0, u1, C, q, rem;
  };
  auto run_of = [&](int per_head) {
    Run r;
    const int units = per_head * HG, b = (int)blockIdx.x;
    r.C = max(1, min(units, (int)gridDim.x));  // CTAs with a run
    r.q = (int)((uint32_t)units / (uint32_t)r.C);
    r.rem = units - r.q * r.C;
    r.u0 = b * r.q + min(b, r.rem);
    r.u1 = b < r.C ? r.u0 + r.q + (b < r.rem ? 1 : 0) : r.u0;
    return r;
  };
  Run run;
  int s0 = 0, before = 0;                      // the run's first sequence, and the tiles (per pair) of those before it
  if (sa.n <= 32 * LANE_SEQS) {                // every warp by itself
    const int K = (sa.n + 31) / 32;
    int t[LANE_SEQS], mine = 0;
#pragma unroll
    for (int i = 0; i < LANE_SEQS; ++i) t[i] = i < K ? pos_of(lane * K + i) : -1;
#pragma unroll
    for (int i = 0; i < LANE_SEQS; ++i) mine += t[i] = tiles_at(t[i]);
    const int end = warp_scan(mine);
    run = run_of(__shfl_sync(0xffffffffu, end, 31));
    const uint32_t past = __ballot_sync(0xffffffffu, (int64_t)end * HG > run.u0);   // (the first of them holds it)
    int at = end - mine, s = lane * K;
#pragma unroll
    for (int i = 0; i < LANE_SEQS; ++i)
      if (i < K && (int64_t)(at + t[i]) * HG <= run.u0) {
        at += t[i];
        ++s;
      } else {
        break;
      }
    const int owner = past ? __ffs(past) - 1 : 0;
    s0 = __shfl_sync(0xffffffffu, s, owner);
    before = __shfl_sync(0xffffffffu, at, owner);
  } else {                                     // the block, THREADS sequences at a time
    auto block_scan = [&](int x, int* total) {
      x = warp_scan(x);
      __syncthreads();
      if (lane == 31) red[warp] = x;
      __syncthreads();
      int head = 0, all = 0;
      for (int w = 0; w < WARPS + PRODUCERS; ++w) {
        if (w < warp) head += red[w];
        all += red[w];
      }
      *total = all;
      return x + head;
    };
    int per_head = 0;
    for (int b = 0; b < sa.n; b += THREADS) {
      int t;
      block_scan(tiles_at(pos_of(b + (int)threadIdx.x)), &t);
      per_head += t;
    }
    run = run_of(per_head);
    if (run.u0 < run.u1) {
      bool there = false;
      for (int b = 0, carry = 0; !there; b += THREADS) {
        int t;
        const int mine = tiles_at(pos_of(b + (int)threadIdx.x)), end = carry + block_scan(mine, &t);
        if ((int64_t)end * HG > run.u0 && (int64_t)(end - mine) * HG <= run.u0) {
          found[0] = b + (int)threadIdx.x;
          found[1] = end - mine;
        }
        carry += t;
        there = (int64_t)carry * HG > run.u0;
      }
      __syncthreads();
      s0 = found[0];
      before = found[1];
    }
  }
  Cursor c0 = {};
  if (run.u0 < run.u1) {
    look_at(c0, s0, pos_of(s0));
    const int r = run.u0 - before * HG;
    c0.hg = r / c0.T;
    c0.t = r - c0.hg * c0.T;
  }
  // runs fn(cursor, tiles of the pair in this run, the next pair's cursor, whether there is one) over the pairs of
  // the run; positions are read 32 sequences at a time
  auto each_pair = [&](auto&& fn) {
    if (run.u0 >= run.u1) return;
    Cursor c = c0;
    int base = c.s + 1, ahead = pos_of(base + lane);
    for (int u = run.u0;;) {
      const int m = min(c.T - c.t, run.u1 - u);
      u += m;
      Cursor nx = c;
      nx.t = 0;
      if (u < run.u1 && ++nx.hg == HG) {       // the next sequence that sees something
        nx.hg = 0;
        uint32_t some;
        while (!(some = __ballot_sync(0xffffffffu, base + lane > c.s && tiles_at(ahead) > 0)) && base < sa.n) {
          base += 32;
          ahead = pos_of(base + lane);
        }
        const int l = __ffs(some) - 1;
        look_at(nx, base + l, __shfl_sync(0xffffffffu, ahead, l));
      }
      if (!fn(c, m, nx, u < run.u1) || u >= run.u1) return;
      c = nx;
    }
  };

  uint32_t filled = 0;         // (producers) per stage: filled (bit st), parity of the last fill (bit 16 + st)
  if (warp >= WARPS) {
    // ---- TMA producers: every third tile each (a warp passes once over its loop for each box, whose operands are
    // uniform: with one warp, or four for a quarter of each tile, the tiles of 16-row pages or 64-byte rows take
    // longer than their bytes)
    constexpr int NB = KIND == E4M3 ? 1 : HD / 64, ROW = KIND == E4M3 ? HD : 128;   // boxes of a page, bytes of a box row
    const int pw = warp - WARPS, plane = lane & 1, box = (lane >> 1) % NB, part = (lane >> 1) / NB;   // this lane's box
    const int npg = pg.shift < 6 ? KT >> pg.shift : 1, br = KT / npg;     // pages of a tile, rows of a box
    int i = 0;
    int cs = -1, blk = -1, cur = 0, ns_ = -1, nblk = -1, next = 0;   // page ids of 32 columns: of a block, and of the next
    each_pair([&](const Cursor& c, int m, const Cursor& nx, bool more) {
      const int head = c.hg / sa.groups, last = (c.v.end - 1) >> pg.shift;
      auto ids = [&](const Cursor& w, int b) {
        const int col = b * 32 + lane;
        return col <= (w.v.end - 1) >> pg.shift ? pg.table[(int64_t)w.s * pg.table_stride + col] : -1;
      };
      auto block_of = [&](const Cursor& w, int t) { return (w.tl.at(t) * KT >> pg.shift) >> 5; };
      const int i0 = i;
      i += m;
      for (int x = (pw - i0 % PRODUCERS + PRODUCERS) % PRODUCERS; x < m; x += PRODUCERS) {
        const int t = c.t + x, j0 = c.tl.at(t) * KT, col = j0 >> pg.shift;
        if (col >> 5 != blk || c.s != cs) {
          cur = ns_ == c.s && nblk == col >> 5 ? next : ids(c, col >> 5);
          cs = c.s;
          blk = col >> 5;
          // the block that comes behind it: of this pair, or the next pair's first
          if (block_of(c, c.t + m - 1) != blk) {
            ns_ = c.s;
            nblk = t < c.tl.head && block_of(c, c.tl.head - 1) == blk ? block_of(c, c.tl.head) : blk + 1;
            next = ids(c, nblk);
          } else if (more) {
            ns_ = nx.s;
            nblk = block_of(nx, 0);
            next = ids(nx, nblk);
          }
        }
        const int id = __shfl_sync(0xffffffffu, cur, (col + part) & 31);
        const int tile = i0 + x, st = tile % NST;
        const bool free = mbar_wait(&empty[st], (tile / NST & 1) ^ 1, abort_flag, &g_given_up);
        if (!__all_sync(0xffffffffu, free ? 1 : 0)) return false;
        const int there = min(npg, last - col + 1);            // pages that the sequence has
        if (lane == 0) mbar_expect_tx(&full[st], (uint32_t)(there * NB * 2 * br * ROW));
        __syncwarp();
        if constexpr (KIND == E4M3) {
          // the tile's scales, 4 rows of a plane a lane (rows without a page: zeros)
          const int sr = 4 * (lane & 15), sp = lane >> 4, spart = sr / br;
          const int sid = __shfl_sync(0xffffffffu, cur, (col + spart) & 31);
          const bool on = spart < there && sid >= 0 && sid < pg.n_pages;
          copy16_async(sm + L::SC + (st * 2 * KT + sp * KT + sr) * 4,
                       pg.scales + ((((int64_t)sp * pg.n_pages + (on ? sid : 0)) * pg.Hkv + head) << pg.shift) +
                           ((j0 + sr) & ((1 << pg.shift) - 1)),
                       on);
          arrive_after_copies(&full[st]);
        }
        filled = (filled & ~(1u << (16 + st))) | 1u << st | (uint32_t)(tile / NST & 1) << (16 + st);
        if (part < there)
          tma5(sm + st * L::TILE + plane * L::PLANE + box * (KT * 128) + part * br * ROW, &map, &full[st], box * 64,
               j0 & ((1 << pg.shift) - 1), head, id, plane);
      }
      return true;
    });
  } else {
    // ---- computing warps: rows 16 sub .. +15 of every second tile, or third with 12 warps
    const int grp = warp >> 2, sub = warp & 3, g = lane >> 2, t4 = lane & 3;
    const float sl2 = a.scale * 1.4426950408889634f;
    float* pub = (float*)(sm + L::OUT);
    float2* ml = (float2*)(sm + L::ML);
    const uint32_t base_k = smem_u32(sm);
    bool ok = true;
    int i = 0;                                 // tiles of the run before the pair
    // tokens that see nothing: zeros
    for (int s = blockIdx.x; s < sa.n; s += gridDim.x)
      if (tiles_at(sa.pos[s]) == 0)
        for (int e = threadIdx.x; e < a.Hq * HD / 8; e += WARPS * 32)
          reinterpret_cast<uint4*>((uint16_t*)a.out + (int64_t)s * a.Hq * HD)[e] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
      Record* rec = reinterpret_cast<Record*>((float*)a.ws + 2 * (int64_t)gridDim.x * slot_floats(HD)) + blockIdx.x;
      rec->valid = 0;
    }
    uint32_t qn[NH][HD / 16][2];               // the next pair's q
    auto load_q = [&](const Cursor& c) {
      const int kvh = c.hg / sa.groups, h0 = kvh * sa.G + (c.hg % sa.groups) * 8 * NH;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        const int r = 8 * nh + g;
        const uint16_t* qp = (const uint16_t*)a.q + (int64_t)c.s * a.q_stride + (int64_t)(h0 + r) * HD;
        const bool there = r < min(8 * NH, (kvh + 1) * sa.G - h0);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = KIND == E4M3 ? 64 * (ks >> 2) + 16 * t4 + 4 * (ks & 3) + 2 * e : 16 * ks + 2 * t4 + 8 * e;
            qn[nh][ks][e] = there ? __ldg(reinterpret_cast<const uint32_t*>(qp + d)) : 0u;
          }
      }
    };
    constexpr bool AHEAD = NH == 1 || HD == 64;   // (the registers of 16 q heads of 128 leave no room)
    if (AHEAD && run.u0 < run.u1) load_q(c0);
    each_pair([&](const Cursor& c, int m, const Cursor& nx, bool more) {
      const int kvh = c.hg / sa.groups, h0 = kvh * sa.G + (c.hg % sa.groups) * 8 * NH;
      const int nq = min(8 * NH, (kvh + 1) * sa.G - h0);       // q heads of the pair
      // Q^T as B fragments: q head 8 nh + g; d of k-step ks as the K operand has it
      uint32_t q[NH][HD / 16][2];
      float qs[NH][2];                                         // what a score of q head 8 nh + 2 t + e is multiplied by
      if constexpr (!AHEAD) load_q(c);
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) q[nh][ks][0] = qn[nh][ks][0], q[nh][ks][1] = qn[nh][ks][1];
        qs[nh][0] = qs[nh][1] = sl2;
        if constexpr (KIND == E4M3 && QBF) {                   // to f16, the head's largest element near 2^14
          uint32_t top = 0;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) top = max(top, max(q[nh][ks][e] & 0x7fffu, q[nh][ks][e] >> 16 & 0x7fffu));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int E = min(max((int)(top >> 7) - 127, -100), 127);
          const float up = __uint_as_float((uint32_t)(14 - E + 127) << 23);
          const float down = sl2 * __uint_as_float((uint32_t)(E - 14 + 127) << 23);
          qs[nh][0] = __shfl_sync(0xffffffffu, down, 8 * t4);  // (of heads 2 t and 2 t + 1)
          qs[nh][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              q[nh][ks][e] = h2u(__uint_as_float(q[nh][ks][e] << 16) * up,
                                 __uint_as_float(q[nh][ks][e] & 0xffff0000u) * up);
        }
      }
      if (AHEAD && more) load_q(nx);                           // (used when this pair has ended)
      float o[NH][HD / 16][4] = {};
      float mx[NH][2], sum[NH][2] = {};                        // base and sum of q heads 8 nh + 2 t + e
      // e4m3: the sum's base (mx: the products'). It is looked at where mx moves; while exponents stay within NEAR that is
      // enough: a move leaves mx - mz <= TOP - HEAD + NEAR, and a later z <= mx + TOP + NEAR is then below mz + 70. Once
      // one did not (wide), it is looked at in every tile
      float mz[NH][2];
      bool wide = false;
      int unit = NO_UNIT;                                      // e4m3: O counts 2^unit, the bound of the first scales seen
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) mx[nh][0] = mx[nh][1] = mz[nh][0] = mz[nh][1] = NO_BASE;
      for (int x = (grp - i % GROUPS + GROUPS) % GROUPS; x < m && ok; x += GROUPS) {
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
          float s[NH][4] = {};                                 // rows key8(g) (0, 1) and 8 + key8(g) (2, 3), heads 2 t + e
          // ---- S^T = K Q^T
          if constexpr (KIND != E4M3) {
            const int r = sub * 16 + (lane & 15), ch = lane >> 4;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
              uint32_t k[4];
              ldsm4<false>(k, kb + (ks >> 2) * (KT * 128) + r * 128 + ((((ks & 3) * 2 + ch) ^ (r & 7)) << 4));
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma16816<PBF>(s[nh], k, q[nh][ks][0], q[nh][ks][1]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < HD / 64; ++j) {
              uint32_t w[2][4];
#pragma unroll
              for (int nb = 0; nb < 2; ++nb) {
                const int r = sub * 16 + nb * 8 + key8<KIND>(g);
                const int ch = HD == 128 ? (4 * j + t4) ^ (r & 7) : t4 ^ (r >> 1 & 3);
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[nb][0]), "=r"(w[nb][1]), "=r"(w[nb][2]), "=r"(w[nb][3])
                             : "r"(kb + r * HD + (ch << 4)));
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t ka[4];
                widen4(w[0][k], ka[0], ka[2]);
                widen4(w[1][k], ka[1], ka[3]);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma16816<false>(s[nh], ka, q[nh][4 * j + k][0], q[nh][4 * j + k][1]);
              }
            }
          }
          // ---- scores in the log2 domain, hidden rows -inf
          bool hid[2] = {false, false};                        // rows key8(g), 8 + key8(g)
          float ks[2] = {1.f, 1.f}, v[2], f[2], ex[2];         // e4m3: K's scale, V's and its fraction and exponent
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int r = b * 8 + key8<KIND>(g), j = j0 + r;
            if (!whole) hid[b] = j >= c.v.end || (j < c.v.lo && j >= c.v.sk);
            if constexpr (KIND == E4M3) {
              const float* sc = (const float*)(sm + L::SC) + st * 2 * KT + sub * 16 + r;
              ks[b] = sc[0];
              v[b] = sc[KT];
            }
          }
          if constexpr (KIND == E4M3) {
            int E[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t u = __float_as_uint(v[b]);
              E[b] = (int)(u >> 23) - 126;
              ex[b] = (float)(E[b] - unit);
              f[b] = __uint_as_float((u & 0x7fffffu) | 126u << 23);
            }
            // a first scale, one far from the unit, or one at or below fp32's smallest normal number
            if (__any_sync(0xffffffffu, min(E[0], E[1]) < max(unit - NEAR, -125) || max(E[0], E[1]) > unit + NEAR)) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (unit == NO_UNIT) {                         // (hidden rows and those of scale 0 have no say)
                  const int top = __reduce_max_sync(0xffffffffu, hid[b] || v[b] == 0.f ? INT_MIN : E[b]);
                  if (top != INT_MIN) unit = top;
                }
              bool far = false;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int rel = max(E[b] - unit, -80), up = -(unit + rel);   // (2^-80 below the unit: the rest stays in f)
                ex[b] = (float)rel;
                f[b] = v[b] * pow2f(up >> 1) * pow2f(up - (up >> 1));
                far |= !hid[b] && (rel < -NEAR || rel > NEAR);
              }
              wide |= __any_sync(0xffffffffu, far) != 0;
            }
          }
          uint32_t p[NH][2];                                   // P^T: rows 2 t, 2 t + 1 of each block, q head g
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            float up[2];                                       // what the base is taken from: score, or score and exponent
            bool move[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float zs = qs[nh][e] * ks[b];
                if constexpr (KIND == E4M3) zs = fminf(zs, 3.402823466e38f);   // (0 x inf of a score of 0)
                s[nh][2 * b + e] = hid[b] ? -INFINITY : s[nh][2 * b + e] * zs;
              }
              if constexpr (KIND == E4M3) up[e] = fmaxf(s[nh][e] + ex[0], s[nh][2 + e] + ex[1]);
              else up[e] = fmaxf(s[nh][e], s[nh][2 + e]);
            }
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
              up[0] = fmaxf(up[0], __shfl_xor_sync(0xffffffffu, up[0], k));
              up[1] = fmaxf(up[1], __shfl_xor_sync(0xffffffffu, up[1], k));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) move[e] = up[e] - mx[nh][e] > TOP;
            if (__any_sync(0xffffffffu, move[0] || move[1] || (KIND == E4M3 && wide))) {
              // where a base at b goes for a maximum x, and what is multiplied by al for it
              auto moved = [](float b, float x) { return x - b > TOP ? (fabsf(x) < FAR ? x - HEAD : x) : b; };
              auto shrink = [](float b, float to) { return b == to ? 1.f : ex2(b - to); };
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float to = moved(mx[nh][e], up[e]), al = shrink(mx[nh][e], to);
                mx[nh][e] = to;
                if constexpr (KIND == E4M3) {
                  float z = fmaxf(s[nh][e], s[nh][2 + e]);
#pragma unroll
                  for (int k = 4; k < 32; k <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, k));
                  const float tz = moved(mz[nh][e], z);
                  sum[nh][e] *= shrink(mz[nh][e], tz);
                  mz[nh][e] = tz;
                } else {
                  sum[nh][e] *= al;
                }
#pragma unroll
                for (int b = 0; b < HD / 16; ++b) {
                  o[nh][b][e] *= al;
                  o[nh][b][2 + e] *= al;
                }
              }
            }
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float base = mx[nh][e], base_z = KIND == E4M3 ? mz[nh][e] : base;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float z = s[nh][2 * b + e], d = ex2(z - base_z);   // (e4m3: the sum's weight)
                sum[nh][e] += d;
                if constexpr (KIND == E4M3) w[2 * b + e] = hid[b] ? 0.f : ex2(z + ex[b] - base) * f[b];
                else w[2 * b + e] = d;
              }
            }
            p[nh][0] = transpose8(pack_w<PBF>(w[0], w[1]));
            p[nh][1] = transpose8(pack_w<PBF>(w[2], w[3]));
          }
          // ---- O^T += V^T P^T; the values of hidden rows are zeros (0 x NaN is not)
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};       // of the rows' pairs key8(2 t), key8(2 t + 1) of each block
          if (!whole) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t bits = __ballot_sync(0xffffffffu, hid[b]);   // (lane 4 n: row n)
              keep[b] = (bits >> (8 * t4) & 1 ? 0u : 0xffffu) | (bits >> (8 * t4 + 4) & 1 ? 0u : 0xffff0000u);
            }
          }
          if constexpr (KIND != E4M3) {
            const int r = sub * 16 + (lane & 7) + (lane & 16 ? 8 : 0), ch = lane >> 3 & 1;
#pragma unroll
            for (int b = 0; b < HD / 16; ++b) {
              uint32_t v[4];
              ldsm4<true>(v, vb + (b >> 2) * (KT * 128) + r * 128 + ((((b & 3) * 2 + ch) ^ (r & 7)) << 4));
              if (!whole) {
                v[0] &= keep[0];
                v[1] &= keep[0];
                v[2] &= keep[1];
                v[3] &= keep[1];
              }
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma16816<PBF>(o[nh][b], v, p[nh][0], p[nh][1]);
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
            if (!whole) {                                      // (a NaN code of a hidden row: bytes of zero)
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int y = 0; y < NW; ++y) w[k][y] &= keep[k >> 1] >> (16 * (k & 1)) & 1 ? 0xffffffffu : 0u;
            }
#pragma unroll
            for (int y = 0; y < NW; ++y)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t y0 = __byte_perm(w[0][y], w[1][y], half ? 0x7362 : 0x5140);
                const uint32_t y1 = __byte_perm(w[2][y], w[3][y], half ? 0x7362 : 0x5140);
                uint32_t v[4];
                widen4(y0, v[0], v[1]);
                widen4(y1, v[2], v[3]);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma16816<false>(o[nh][2 * y + half], v, p[nh][0], p[nh][1]);
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      i += m;
      // ---- the pair ends here: the warps' sums through shared memory, 8 q heads at a time
      const bool starts = c.t == 0, ends = c.t + m == c.T;
      float* slot = (float*)a.ws + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * slot_floats(HD);
#pragma unroll
      for (int half = 0; half < NH; ++half) {
        if (8 * half >= nq) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = sum[half][e];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
          const float m0 = KIND == E4M3 ? mz[half][e] : mx[half][e], m1 = m0 == NO_BASE ? -INFINITY : m0;
          if (g == 0) ml[warp * 8 + 2 * t4 + e] = KIND == E4M3 ? leveled(m1, l) : make_float2(m1, l);
          float* at = pub + (warp * 8 + 2 * t4 + e) * L::OSTR;
          if (8 * half + 2 * t4 + e >= nq) continue;           // (no such q head)
          if constexpr (KIND == E4M3) {
            // O counts 2^(unit + mx - mz) beside the sum: half of it at a time, which fp32 holds
            const bool some = l != 0.f && unit != NO_UNIT;
            const float inv = some ? 1.f / l : 0.f, u = some ? ex2(0.5f * (mx[half][e] - mz[half][e] + (float)unit)) : 0.f;
#pragma unroll
            for (int b = 0; b < HD / 16; ++b) {
              o[half][b][e] = o[half][b][e] * inv * u * u;
              o[half][b][2 + e] = o[half][b][2 + e] * inv * u * u;
            }
          }
#pragma unroll
          for (int b = 0; b < HD / 16; ++b) {
            at[out_col<HD, KIND>(b, g, 0)] = o[half][b][e];
            at[out_col<HD, KIND>(b, g, 1)] = o[half][b][2 + e];
          }
        }
        group_sync<WARPS * 32>();
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
            const float wo = KIND == E4M3 ? wt * z.y * SHARE : wt;
            y.x += wo * v.x;
            y.y += wo * v.y;
            y.z += wo * v.z;
            y.w += wo * v.w;
          }
          if constexpr (KIND == E4M3) {                        // a mean again
            const float inv = lsum == 0.f ? 0.f : UNSHARE / lsum;
            y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
          }
          if (starts && ends) {
            const float inv = KIND == E4M3 ? 1.f : lsum == 0.f ? 0.f : 1.f / lsum;
            *reinterpret_cast<uint2*>((uint16_t*)a.out + ((int64_t)c.s * a.Hq + h0 + 8 * half + r) * HD + cv * 4) =
                make_uint2(pack_w<QBF>(y.x * inv, y.y * inv), pack_w<QBF>(y.z * inv, y.w * inv));
          } else {
            *reinterpret_cast<float4*>(slot + (8 * half + r) * HD + cv * 4) = y;
            if (cv == 0) reinterpret_cast<float2*>(slot + 16 * HD)[8 * half + r] = make_float2(M, lsum);
          }
        }
        group_sync<WARPS * 32>();
      }
      if (ends && !starts && threadIdx.x == 0) {
        // the pair's first tile: list position u0 - c.t (this is the run's first pair, the only one it does not
        // start), and the CTA whose run holds it
        const int at = run.u0 - c.t, more = run.rem * (run.q + 1);
        const int f = at < more ? at / (run.q + 1) : run.rem + (at - more) / run.q;
        Record* rec = reinterpret_cast<Record*>((float*)a.ws + 2 * (int64_t)gridDim.x * slot_floats(HD)) + blockIdx.x;
        *rec = Record{c.s, c.hg, f, 1};
      }
      return true;
    });
  }
  __syncthreads();
  if (warp >= WARPS && *abort_flag)            // nothing in flight when the CTA leaves
    for (int st = warp - WARPS; st < NST; st += PRODUCERS)
      if (filled >> st & 1) mbar_drain(&full[st], filled >> (16 + st) & 1);
}

// Joins the parts of the pair that CTA blockIdx.x of the step ended: slot 2 first + 1, then slots 2 c of the CTAs
// behind it. Block y takes rows y, y + gridDim.y, ...; its warps take the parts in turn, and their sums are joined in
// order.
constexpr int JWARPS = 8;
template <int HD, bool QBF, int NH, bool MEANS>
__global__ void __launch_bounds__(JWARPS * 32) join_kernel(const __grid_constant__ StepArgs sa, int C) {
  __shared__ float4 py[JWARPS][32];
  __shared__ float2 pml[JWARPS];
  allow_dependents();
  wait_prerequisites();
  const float* ws = (const float*)sa.a.ws;
  const Record rec = reinterpret_cast<const Record*>(ws + 2 * (int64_t)C * slot_floats(HD))[blockIdx.x];
  if (!rec.valid) return;
  const int kvh = rec.hg / sa.groups, h0 = kvh * sa.G + (rec.hg % sa.groups) * 8 * NH;
  const int nq = min(8 * NH, (kvh + 1) * sa.G - h0);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, parts = (int)blockIdx.x - rec.first + 1;
  for (int r = blockIdx.y; r < nq; r += gridDim.y) {
    float M = -INFINITY, l = 0.f;
    float4 y = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int p = w; p < parts; p += JWARPS) {
      const float* slot = ws + (p == 0 ? 2 * (int64_t)rec.first + 1 : 2 * (int64_t)(rec.first + p)) * slot_floats(HD);
      const float2 z = __ldcg(reinterpret_cast<const float2*>(slot + 16 * HD) + r);
      const float4 v = lane < HD / 4 ? __ldcg(reinterpret_cast<const float4*>(slot + r * HD) + lane)
                                     : make_float4(0, 0, 0, 0);
      if (z.x == -INFINITY && z.y == 0.f) continue;
      const float N = fmaxf(M, z.x), a0 = M == N || l == 0.f ? 1.f : ex2(M - N), a1 = z.x == N ? 1.f : ex2(z.x - N);
      M = N;
      l = a0 * l + a1 * z.y;
      const float wo = MEANS ? a1 * z.y * SHARE : a1;
      y = make_float4(a0 * y.x + wo * v.x, a0 * y.y + wo * v.y, a0 * y.z + wo * v.z, a0 * y.w + wo * v.w);
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
      const float inv = s == 0.f ? 0.f : (MEANS ? UNSHARE : 1.f) / s;
      *reinterpret_cast<uint2*>((uint16_t*)sa.a.out + ((int64_t)rec.seq * sa.a.Hq + h0 + r) * HD + lane * 4) =
          make_uint2(pack_w<QBF>(o.x * inv, o.y * inv), pack_w<QBF>(o.z * inv, o.w * inv));
    }
    __syncthreads();
  }
}

template <int HD, int KIND, bool QBF, int NH>
cudaError_t launch(const StepArgs& sa, int num_sms, cudaStream_t st) {
  using L = Lay<HD, KIND, NH>;
  CUtensorMap map;
  if (!pages_map(&map, sa.a.pages, std::min(KT, 1 << sa.a.pages.shift))) return cudaErrorInvalidValue;
  CK_RET(cudaFuncSetAttribute(step_kernel<HD, KIND, QBF, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  CK_RET(launch_pdl(step_kernel<HD, KIND, QBF, NH>, dim3((unsigned)num_sms), dim3(L::THREADS), L::BYTES, st, map, sa));
  return launch_pdl(join_kernel<HD, QBF, NH, KIND == E4M3>, dim3((unsigned)num_sms, 4), dim3(JWARPS * 32), 0, st, sa,
                    num_sms);
}
template <int HD, int KIND, bool QBF>
cudaError_t launch_nh(const StepArgs& sa, int num_sms, cudaStream_t st) {
  return sa.G <= 8 ? launch<HD, KIND, QBF, 1>(sa, num_sms, st) : launch<HD, KIND, QBF, 2>(sa, num_sms, st);
}
template <int HD>
cudaError_t launch_kind(const StepArgs& sa, int num_sms, cudaStream_t st) {
  if (sa.a.pages.format == KVF_F16) return launch_nh<HD, F16, false>(sa, num_sms, st);
  if (sa.a.pages.format == KVF_BF16) return launch_nh<HD, BF16, true>(sa, num_sms, st);
  return sa.a.bf16 ? launch_nh<HD, E4M3, true>(sa, num_sms, st) : launch_nh<HD, E4M3, false>(sa, num_sms, st);
}
}  // namespace pgs

cudaError_t attention_step_gave_up_word(uint64_t** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), pgs::g_given_up);
}

int64_t attention_paged_step_ws_bytes(int hd, int num_sms) {
  return (int64_t)num_sms * (2 * pgs::slot_floats(hd) * 4 + (int64_t)sizeof(pgs::Record));
}

cudaError_t launch_attention_paged_step(const PagedAttnArgs& a, int n, const int* pos, int num_sms, cudaStream_t st) {
  pgs::StepArgs sa{a, pos, n, a.Hq / a.pages.Hkv, 0, 0};
  sa.groups = sa.G <= 8 ? 1 : (sa.G + 15) / 16;
  sa.HG = sa.groups * a.pages.Hkv;
  return a.pages.hd == 128 ? pgs::launch_kind<128>(sa, num_sms, st) : pgs::launch_kind<64>(sa, num_sms, st);
}

}  // namespace s1
