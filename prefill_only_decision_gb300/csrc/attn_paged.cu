// Attention of prompts over a paged K/V cache, with a sliding window and sinks, on the 5th-generation tensor cores.
//
// Query row i of sequence s, at position p, sees the cached rows j <= p with p - j < window or j < sinks: o =
// softmax(scale q.k) v. The rows of a sequence and the G = Hq / Hkv q heads that share a kv head are packed into
// tiles of 128 matrix rows, RT = floor(128 / G) query rows x G heads. An item is (sequence, tile or two neighbouring
// tiles, kv head) with the 128-key tiles that its rows see: the sinks' and the window's. Its key tiles are split over
// `ns` CTAs, one choice per sequence, when that shortens the call, and combine_kernel joins their (o, m, l) in an
// order that the sizes fix.
//
// One pass over the keys with a running base (near the maximum) and sum in fp32, in two streams of S = Q K^T,
// softmax, O += P V that share the tensor cores: two query tiles over the same key tiles, or one query tile over the
// even and the odd key tiles, joined at the end. A stream takes a key tile in two halves of 64 keys with S in TMEM
// columns of their own, so that products run while the softmax works on the other half. One CTA per SM, 16 warps (19
// with e4m3 pages):
//   warps 0, 15 TMA producers: Q and K, and V: a page box (page x 64 elements) per lane, page ids asked for a tile
//               ahead (one warp for both: 16-row pages 450 us where 32-row ones took 376)
//   warps 1, 14 MMA issue of stream 0 and 1
//   warps 2-5, 6-9  softmax of stream 0, 1: one thread per row (TMEM lane), 64 scores in registers, a lazy rescale
//               of O; P goes back into the TMEM columns of S and is the A operand of O += P V from there
//   warps 10-13 scan the value tiles that hold rows which some query does not see: a hidden row's weight is an exact
//               zero, but 0 x NaN is not, so non-finite elements there become 0 and an item's end adds them to the
//               rows that do see them. (Rows behind a sequence's end and pages that are not loaded are such rows.)
//               With e4m3 pages they widen the K tiles instead and warps 15-18 the V tiles, codes from memory through
//               registers.
// CTAs stay and take items in rounds, the longest first: the next item's Q, K and V are on their way while the last
// one's sums leave (a CTA per item: 16476 rows, window 2048, 240 us; so 202).
// e4m3 pages: the operands are f16, code x scale x 2^(7 - E), E a bound of the scales' exponents (K: of the tile; V:
// running, so that O keeps one unit, rescaled when the bound grows): scales of any size fit f16, and a row 2^-27
// below the largest keeps its code's bits. bf16 queries over them become f16 by a power of two per row. Every
// mbarrier wait is bounded; on expiry an error word is set and every role leaves.
#include <algorithm>
#include <climits>
#include <type_traits>
#include <vector>

#include <cuda_fp8.h>

#include "paged.cuh"

namespace s1 {
namespace pgp {
using namespace t5;
using namespace pga;

constexpr int BQ = 128, BKV = 128, TAB_SMALL = 64, TAB_LARGE = 1024;
enum Kind { F16 = 0, BF16 = 1, E4M3 = 2, E4M3_QBF = 3 };
constexpr bool is_e4m3(int kind) { return kind >= E4M3; }
constexpr bool out_bf16(int kind) { return kind == BF16 || kind == E4M3_QBF; }
constexpr int threads_of(int kind) { return (is_e4m3(kind) ? 19 : 16) * 32; }
constexpr int TMEM_COLS = 512;               // S of stream x at 128 x, O at 256 + 128 x
constexpr int T_O = 256;
constexpr int ITEMS = 18;                    // of a CTA's items, kept in shared memory (later ones: made in their turn)
constexpr int BASES = 16;                    // tiles whose exponent bounds are kept (more than are ever in flight)

__device__ uint64_t g_given_up;              // when a bounded wait last gave up, per device; never cleared

// Sequences of one launch, by value (a captured graph keeps its own copy), those with split items first.
template <int N>
struct Tab {
  int n, split;                // sequences; CTAs of the split ones
  int start[N + 1];            // first CTA of a sequence
  int tiles[N + 1];            // query tiles x kv heads of the split sequences before it
  int row0[N], pos0[N], len[N], seq[N], ns[N];
};
struct Plan {
  int G, RT, nt;               // q heads per kv head, query rows per tile, tiles per item
};

template <int HD>
struct Lay {
  static constexpr int TILE = BKV * HD * 2;
  static constexpr int F = HD == 128 ? 5 : 7, FR = 3;     // stages of both streams' ring, or of each stream's own; odd
  static constexpr int Q = 0;                             // per tile HD/64 boxes of [128 rows][128 B]
  static constexpr int KV2 = Q + 2 * BQ * HD * 2;         // stages with two query tiles
  static constexpr int KV1 = Q + BQ * HD * 2;             // with one
  static constexpr int QSC = KV2 + F * TILE;              // [2][128] floats: what a row's q was divided by
  static constexpr int BASE = QSC + 2 * BQ * 4;           // [2][BASES] exponent bounds
  static constexpr int TABLE = BASE + (2 * BASES + 16) * 4;       // the CTA's first ITEMS items
  static constexpr int BAR = TABLE + ITEMS * 64;
  static constexpr int NS = 2 * FR > F ? 2 * FR : F;
  static constexpr int NBAR = 3 + 4 * NS + 12 + 2 + 2 + 4;
  static constexpr int USED = BAR + NBAR * 8 + 16;
  static_assert(USED <= 227 * 1024, "shared memory of one CTA");
  // above half an SM: each CTA allocates all of TMEM, so two never share one
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr int OSTR = HD + 4;                     // floats per row of a stream's published sums
  static_assert(KV1 + 2 * FR * TILE <= QSC, "both rings fit");
  static_assert(BQ * OSTR * 4 <= 2 * FR * TILE, "published sums fit the K/V stages");
  static_assert(F % 2 == 1 && FR % 2 == 1, "a slot holds K and V tiles in turn");
};

// A stage of the ring of K and V tiles K_0, V_0, K_1, ... With two query tiles both streams read one ring; with one,
// each stream has its own, of its tiles: a parity wait must never run more than one phase ahead of a slot, nor behind
// it. For that K and V fills have barriers of their own, too: who waits for one kind does not see the other's phases.
struct Slot {
  int s;
  uint32_t ph, kind_ph;        // parity of this fill, and of it among the slot's fills of its kind (they take turns)
};
// (both: the ring of both streams; else stream x's; k: the tile's number in the ring)
template <int F, int FR>
__device__ __forceinline__ Slot slot_of(bool both, int x, int k, bool is_v) {
  const uint32_t i = 2 * (uint32_t)k + (is_v ? 1 : 0);
  if (both) return {(int)(i % F), i / F & 1, i / F >> 1 & 1};
  return {(x ? FR : 0) + (int)(i % FR), i / FR & 1, i / FR >> 1 & 1};
}

template <bool BF>
__device__ __forceinline__ bool nonfinite2(uint32_t x) {   // either element of the pair
  constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
  return (x & E) == E || (x >> 16 & E) == E;
}
template <bool BF>
__device__ __forceinline__ uint32_t drop_nonfinite2(uint32_t x) {
  constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
  if ((x & E) == E) x &= 0xffff0000u;
  if ((x >> 16 & E) == E) x &= 0xffffu;
  return x;
}
template <bool BF>
__device__ __forceinline__ bool drop_nonfinite(uint4& x) {   // true: there was one
  if (!(nonfinite2<BF>(x.x) || nonfinite2<BF>(x.y) || nonfinite2<BF>(x.z) || nonfinite2<BF>(x.w))) return false;
  x = make_uint4(drop_nonfinite2<BF>(x.x), drop_nonfinite2<BF>(x.y), drop_nonfinite2<BF>(x.z), drop_nonfinite2<BF>(x.w));
  return true;
}

// Eight e4m3 codes times f to f16. FAST: f is an f16 value.
template <bool FAST>
__device__ __forceinline__ uint4 codes_to_half(const uint2 c, float f) {
  uint32_t h[4];
  widen4(c.x, h[0], h[1]);
  widen4(c.y, h[2], h[3]);
  const __half2 f2 = __float2half2_rn(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = *reinterpret_cast<const __half2*>(&h[i]);
    if constexpr (FAST) {
      const __half2 y = __hmul2(x, f2);
      h[i] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const float2 z = __half22float2(x);
      h[i] = h2u(z.x * f, z.y * f);
    }
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// The four warps of a plane's loaders.
__device__ __forceinline__ void plane_sync(int plane) {
  if (plane) asm volatile("bar.sync 2, 128;" ::: "memory");
  else asm volatile("bar.sync 1, 128;" ::: "memory");
}

// The exponent bound of a scale: scale < 2^E (subnormal ones: 2^-126). Scales that are not finite or not there have none.
constexpr int NO_BOUND = -1000;
__device__ __forceinline__ int bound_of(float scale) {
  const uint32_t u = __float_as_uint(scale);
  return u == 0 || (u >> 23) >= 255 ? NO_BOUND : (int)(u >> 23) - 126;
}

// One of a CTA's items: (sequence, one or two query tiles, kv head) and a part of its key tiles.
struct alignas(16) Item {
  int w, ns, g, two;           // number in the list, parts of the sequence's items, kv head, is there a second query tile
  int row0, seq, v0, v1;       // the sequence's first row of q, its row of the table; the item's first row, one past its last
  int pos0, lo, sk, n;         // position of the sequence's first row; some row sees: [0, sk) and [lo, end()); key tiles
  int head, sink0, tail0, pad;   // tile t: t < head: sink0 + t, else tail0 + t
  __device__ int p_first() const { return pos0 + v0; }
  __device__ int end() const { return pos0 + v1; }
  __device__ int tile(int t) const { return (t + (t < head ? sink0 : tail0)) * BKV; }
  // a key tile that some query row does not see in full
  __device__ bool partly(int j0, int window, int sinks) const {
    return j0 + BKV - 1 > p_first() || (window && end() - 1 - j0 >= window && j0 + BKV > sinks);
  }
};
template <int N>
__device__ __forceinline__ Item item_of(const Tab<N>& tab, const PagedAttnArgs& a, const Plan& pl, int w) {
  Item it;
  int si = 0;
  for (int hi = tab.n - 1; si < hi;) {
    const int mid = (si + hi + 1) >> 1;
    if (tab.start[mid] <= w) si = mid;
    else hi = mid - 1;
  }
  const int len = tab.len[si], MT = (len + pl.RT - 1) / pl.RT, MP = (MT + pl.nt - 1) / pl.nt;
  it.w = w;
  it.ns = tab.ns[si];
  it.row0 = tab.row0[si];
  it.seq = tab.seq[si];
  it.pos0 = tab.pos0[si];
  // whole items: the last rows, which see most, first; parts: the items that read the same keys side by side
  const int local = w - tab.start[si], part = it.ns > 1 ? local / (MP * a.pages.Hkv) : 0;
  const int item = local - part * MP * a.pages.Hkv, a0 = it.ns > 1 ? MP : a.pages.Hkv;
  const int q = item / a0, r = item - q * a0;
  it.g = it.ns > 1 ? q : r;
  const int mp = MP - 1 - (it.ns > 1 ? r : q);
  it.two = pl.nt == 2 && 2 * mp + 1 < MT;
  it.v0 = pl.nt * mp * pl.RT;
  it.v1 = min(len, it.v0 + (it.two ? 2 : 1) * pl.RT);
  Seen all;
  all.end = it.end();
  all.lo = a.window && it.p_first() - (a.window - 1) > 0 ? it.p_first() - (a.window - 1) : 0;
  all.sk = min(a.sinks, all.lo);
  it.lo = all.lo;
  it.sk = all.sk;
  const Tiles tl = tiles_of<BKV>(all);
  const int total = tl.count(), per = (total + it.ns - 1) / it.ns, jb = min(total, part * per);
  it.n = min(total, jb + per) - jb;
  it.head = tl.head - jb;
  it.sink0 = jb;
  it.tail0 = tl.first - tl.head + jb;
  it.pad = 0;
  return it;
}

// Adds the non-finite elements of columns c .. c + CW - 1 of the partly hidden value rows that a query sees.
template <bool E4, bool PBF, int CW>
__device__ __forceinline__ void add_nonfinite(const Item& it, const PagedAttnArgs& a, int pos, int row_lo, int c,
                                              uint32_t* o) {
  const PagesArgs& pg = a.pages;
  auto add = [](uint32_t& x, float y) { x = __float_as_uint(__uint_as_float(x) + y); };
  for (int t = 0; t < it.n; ++t) {
    const int j0 = it.tile(t);
    if (!it.partly(j0, a.window, a.sinks)) continue;
    for (int j = j0; j < j0 + BKV && j <= pos; ++j) {
      if (j < row_lo && j >= a.sinks) continue;
      const int id = pg.table[(int64_t)it.seq * pg.table_stride + (j >> pg.shift)];
      if (id < 0 || id >= pg.n_pages) continue;
      const int64_t vec = (((pg.n_pages + (int64_t)id) * pg.Hkv + it.g) << pg.shift) + (j & ((1 << pg.shift) - 1));
      if constexpr (E4) {
#pragma unroll
        for (int e = 0; e < CW; ++e) {
          const __nv_fp8_storage_t code = ((const __nv_fp8_storage_t*)pg.data)[vec * pg.hd + c + e];
          const float y = __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))) * pg.scales[vec];
          if (!isfinite(y)) add(o[e], y);
        }
      } else {
        const uint4* at = reinterpret_cast<const uint4*>((const uint16_t*)pg.data + vec * pg.hd + c);
#pragma unroll
        for (int e = 0; e < CW / 8; ++e) {
          const uint4 y = at[e];
          const uint32_t y4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (nonfinite2<PBF>(y4[i])) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint16_t raw = (uint16_t)(y4[i] >> (16 * z));
                const float f = PBF ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw));
                if (!isfinite(f)) add(o[8 * e + 2 * i + z], f);
              }
            }
        }
      }
    }
  }
}

template <int HD, int KIND, int N>
__global__ void __launch_bounds__(threads_of(KIND), 1)
    paged_kernel(const __grid_constant__ Tab<N> tab, const __grid_constant__ CUtensorMap mapKV,
                 const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ PagedAttnArgs a, const Plan pl) {
  using L = Lay<HD>;
  constexpr bool E4 = is_e4m3(KIND), PBF = KIND == BF16, OBF = out_bf16(KIND), QTMA = KIND != E4M3_QBF;
  constexpr int NB = HD / 64, F = L::F, FR = L::FR, NS = L::NS;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = (uint64_t*)(sm + L::BAR);
  uint64_t* q_full = bars;                     // an item's Q is there
  uint64_t* q_empty = bars + 1;                // its products have read it
  uint64_t* kv_free = bars + 2;                // (one query tile) the published sums in the K/V stages are read
  uint64_t* full = bars + 3;                   // [NS] a K tile is there
  uint64_t* vfull = full + NS;                 // [NS] a V tile is there
  uint64_t* empty = vfull + NS;                // [NS]
  uint64_t* ready = empty + NS;                // [NS] the V tile is scanned (not with e4m3)
  uint64_t* s_full = ready + NS;               // [2 streams][2 halves of the key tile]
  uint64_t* p_full = s_full + 4;               // [2][2]
  uint64_t* o_step = p_full + 4;               // [2][2] the half's P V has completed
  uint64_t* o_done = o_step + 4;               // [2] the stream's last product of an item has completed
  uint64_t* mma_idle = o_done + 2;             // [2]
  uint64_t* joined = mma_idle + 2;             // [4 quadrants] stream 1's sums are published
  uint32_t* tmem_slot = (uint32_t*)(bars + L::NBAR);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* v_flag = (volatile int*)(tmem_slot + 2);   // a value of a partly hidden tile is not finite
  volatile int* base_k = (volatile int*)(sm + L::BASE);    // [BASES] by tile
  volatile int* base_v = base_k + BASES + 16;              // (between them the loaders' bounds)

  const PagesArgs& pg = a.pages;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const bool pair = pl.nt == 2;                // two query tiles share the ring; else one's key tiles alternate
  if (threadIdx.x == 0) {
    mbar_init(q_full, QTMA ? 1 : 8);
    mbar_init(q_empty, 2);
    mbar_init(kv_free, 4);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], E4 ? 4 : 1);
      mbar_init(&vfull[s], E4 ? 4 : 1);
      mbar_init(&empty[s], pair ? 2 : 1);      // the streams that read the slot
      mbar_init(&ready[s], 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&mma_idle[x], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[2 * x + h], 1);
        mbar_init(&p_full[2 * x + h], 4);
        mbar_init(&o_step[2 * x + h], 1);
      }
      mbar_init(&o_done[x], 1);
    }
    for (int x = 0; x < 4; ++x) mbar_init(&joined[x], 1);
    *abort_flag = 0;
    *v_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<TMEM_COLS>(tmem_slot);
  // every gridDim-th item of the list, there and back again, so that a list that grows cheaper stays even
  const int listed = tab.start[tab.n];
  auto number_of = [&](int k) { return k * (int)gridDim.x + (int)(k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
  const int rounds = (listed + (int)gridDim.x - 1) / (int)gridDim.x;
  const int items = rounds - (number_of(rounds - 1) >= listed ? 1 : 0);
  Item* table = reinterpret_cast<Item*>(sm + L::TABLE);
  if (threadIdx.x >= 64 && (int)threadIdx.x - 64 < min(items, ITEMS))
    table[threadIdx.x - 64] = item_of(tab, a, pl, number_of((int)threadIdx.x - 64));
  allow_dependents();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  uint8_t* kvst = sm + (pair ? L::KV2 : L::KV1);
  auto wwait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_given_up) ? 1 : 0) != 0;
  };
  // This CTA's items: fn(item, its number, tiles before it of stream 0 and of stream 1) until it returns false.
  auto item_at = [&](int k) { return k < ITEMS ? table[k] : item_of(tab, a, pl, number_of(k)); };
  auto each_item = [&](auto&& fn) {
    int t0 = 0, t1 = 0;
    for (int k = 0; k < items; ++k) {
      const Item it = item_at(k);
      if (!fn(it, k, t0, t1)) break;
      t0 += pair ? it.n : (it.n + 1) >> 1;
      t1 += pair ? (it.two ? it.n : 0) : it.n >> 1;
    }
  };
  // an item's tile t in the ring: the stream whose ring it is (pair: 0), and its number there
  auto slot = [&](int t, bool is_v, int t0, int t1) {
    return pair ? slot_of<F, FR>(true, 0, t0 + t, is_v) : slot_of<F, FR>(false, t & 1, (t & 1 ? t1 : t0) + (t >> 1), is_v);
  };
  uint32_t done = 0;           // (producers) per slot: begun (bit s), parity of the last fill of their kind (bit 16 + s)
  int q_done = 0;              // (producer) Q fills
  if (warp == 0 || (!E4 && warp == 15)) {
    // ---- TMA producers: Q, and with 16-bit pages the K tiles and (warp 15) the V tiles. A producer sees every
    // second fill of a slot only; a parity wait needs all fills but the last to be over, and they are: the producer's
    // own last tile came after the consumption of an item behind those.
    wait_prerequisites();
    const bool is_v = warp == 15;
    uint64_t* bar = is_v ? vfull : full;
    const int npg = BKV >> pg.shift, box = lane % NB, pp = lane / NB;
    each_item([&](const Item& it, int k, int t0, int t1) {
      if (QTMA && !is_v) {
        if (!wwait(q_empty, (k & 1) ^ 1)) return false;
        const int tiles = it.two ? 2 : 1;
        if (lane == 0) mbar_expect_tx(q_full, (uint32_t)(tiles * NB * pl.G * pl.RT * 128));
        __syncwarp();
        if (lane < tiles * NB)
          tma3(sm + L::Q + (lane / NB) * (BQ * HD * 2) + (lane % NB) * (BQ * 128), &mapQ, q_full, 64 * (lane % NB),
               it.g * pl.G, it.row0 + it.v0 + (lane / NB) * pl.RT);
        q_done = k + 1;
      }
      if constexpr (E4) return true;
      if (!pair && k > 0 && !wwait(kv_free, (k - 1) & 1)) return false;
      const int last = (it.end() - 1) >> pg.shift;
      const int64_t trow = (int64_t)it.seq * pg.table_stride;
      auto page_id = [&](int t) {              // of this lane's part of tile t
        if (t >= it.n || pp >= npg) return -1;
        const int col = (it.tile(t) >> pg.shift) + pp;
        return col <= last ? pg.table[trow + col] : -1;
      };
      int next = page_id(0);                   // asked for a tile ahead
      for (int t = 0; t < it.n; ++t) {
        const Slot sl = slot(t, is_v, t0, t1);
        const int s = sl.s, j0 = it.tile(t), id = next;
        next = page_id(t + 1);
        if (!wwait(&empty[s], sl.ph ^ 1)) return false;
        const int there = min(npg, last - (j0 >> pg.shift) + 1);   // pages that the sequence has
        if (lane == 0) mbar_expect_tx(&bar[s], (uint32_t)(there << pg.shift) * (HD * 2));
        __syncwarp();
        if (pp < there)
          tma5(kvst + s * L::TILE + box * (BKV * 128) + (pp << pg.shift) * 128, &mapKV, &bar[s], 64 * box, 0, it.g, id,
               is_v ? 1 : 0);
        done = (done & ~(1u << (16 + s))) | 1u << s | sl.kind_ph << (16 + s);
      }
      return true;
    });
  } else if (warp == 1 || warp == 14) {
    // ---- MMA issue of stream x: the whole warp waits, one lane issues. A stream's products run in
    // the order they are issued, so S of its next tile may take the columns that P V reads before it
    const int x = warp == 1 ? 0 : 1;
    const bool leader = elect_one();
    constexpr uint32_t ID_S = idesc_f16(BKV / 2, PBF, 0, 0), ID_O = idesc_f16(HD, PBF, 0, 1);
    const uint32_t tS = tmem + x * 128, tO = tmem + T_O + x * 128;
    const uint64_t qd = desc_sw128(smem_u32(sm + L::Q) + (pair && x ? BQ * HD * 2 : 0), 16);
    auto scores = [&](int h, int s) {          // S = Q K^T over half h of the tile in slot s
      const uint64_t kd = desc_sw128(smem_u32(kvst + s * L::TILE) + h * (BKV / 2 * 128), 16);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
        mma_ss(tS + h * (BKV / 2), qd + (uint64_t)(((kk >> 2) * (BQ * 128) + (kk & 3) * 32) >> 4), kd + off, ID_S,
               kk > 0 ? 1u : 0u);
      }
      commit(&s_full[2 * x + h]);
    };
    auto values = [&](int h, int s, bool acc) {   // O += P V over half h
      const uint64_t vd = desc_sw128(smem_u32(kvst + s * L::TILE) + h * (BKV / 2 * 128), BKV * 128);
#pragma unroll
      for (int kk = 0; kk < BKV / 32; ++kk)
        mma_ts(tO, tS + h * (BKV / 2) + kk * 8, vd + (uint64_t)(kk * 16 * 128 >> 4), ID_O, (acc || kk > 0) ? 1u : 0u);
      commit(&o_step[2 * x + h]);
    };
    wait_prerequisites();                      // (a bounded wait must not begin while the calls before still run)
    each_item([&](const Item& it, int k, int t0, int t1) {
      if (pair && x && !it.two) {              // no second tile: its share of the stages' release
        if (!wwait(q_full, k & 1)) return false;   // (an arrival must not count for the item before)
        if (lane == 0) mbar_arrive(q_empty);
        for (int t = 0; t < 2 * it.n; ++t) {
          const Slot sl = slot(t >> 1, t & 1, t0, t1);
          if (!wwait(t & 1 ? &vfull[sl.s] : &full[sl.s], sl.kind_ph)) return false;
          if (lane == 0) mbar_arrive(&empty[sl.s]);
        }
        return true;
      }
      // of each half h: P V of tile i - 1, then S of tile i into the same columns
      const int cnt = pair ? it.n : (it.n + 1 - x) >> 1, before = x ? t1 : t0;
      if (!wwait(q_full, k & 1)) return false;
      if (cnt == 0 && lane == 0) mbar_arrive(q_empty);
      fence_after();
      for (int i = 0; cnt > 0 && i <= cnt; ++i) {
        const int t = pair ? i : 2 * i + x;
        const Slot ks = slot(t, false, t0, t1);                          // (unused at i = cnt)
        const Slot vs = slot(t - (pair ? 1 : 2), true, t0, t1);          // (unused at i = 0)
        auto half = [&](auto hc) {
          constexpr int h = decltype(hc)::value;
          if (i > 0) {
            if (h == 0 && (!wwait(&vfull[vs.s], vs.kind_ph) || (!E4 && !wwait(&ready[vs.s], vs.kind_ph)))) return false;
            if (!wwait(&p_full[2 * x + h], (before + i - 1) & 1)) return false;
            fence_after();
            if (leader) {
              values(h, vs.s, h > 0 || i > 1);
              if (h) commit(&empty[vs.s]);
              if (h && i == cnt) commit(&o_done[x]);
            }
            __syncwarp();
          }
          if (i < cnt) {
            if (h == 0) {
              if (!wwait(&full[ks.s], ks.kind_ph)) return false;
              fence_after();
            }
            if (leader) {
              scores(h, ks.s);
              if (h) commit(&empty[ks.s]);
              if (h && i == cnt - 1) commit(q_empty);
            }
            __syncwarp();
          }
          return true;
        };
        if (!half(std::integral_constant<int, 0>{}) || !half(std::integral_constant<int, 1>{})) return false;
      }
      return true;
    });
    if (leader) {
      commit(&mma_idle[x]);
      mbar_drain(&mma_idle[x], 0);             // every MMA issued above has completed
    }
  } else if (warp >= 10) {
    const int lw = warp < 14 ? warp - 10 : warp - 15;
    wait_prerequisites();
    if constexpr (!E4) {
      // ---- scan of the partly hidden V tiles: rows 32 lw .. +31. Magnitudes' maximum first; a tile with something
      // that is not finite (rare) once more, to take it out
      constexpr int CH = HD / 8, RPI = 32 / CH, PASSES = 32 / RPI;
      const int c = lane % CH;
      each_item([&](const Item& it, int, int t0, int t1) {
        for (int t = 0; t < it.n; ++t) {
          const Slot k = slot(t, true, t0, t1);
          if (!wwait(&vfull[k.s], k.kind_ph)) return false;
          const int j0 = it.tile(t);
          if (it.partly(j0, a.window, a.sinks)) {
            uint8_t* tile = kvst + k.s * L::TILE;
            auto at = [&](int p) {
              const int r = lw * 32 + p * RPI + lane / CH;
              return reinterpret_cast<uint4*>(tile + (c >> 3) * (BKV * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            };
            using T = std::conditional_t<PBF, bf16, f16>;
            uint32_t top = 0;
#pragma unroll
            for (int p = 0; p < PASSES; p += 8) {
              uint4 y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (p + i < PASSES) y[i] = *at(p + i);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (p + i < PASSES)
                  top = absmax2(T(), top, absmax2(T(), absmax2(T(), y[i].x, y[i].y), absmax2(T(), y[i].z, y[i].w)));
            }
            if (__any_sync(0xffffffffu, nonfinite2<PBF>(top))) {
              bool bad = false;
#pragma unroll 1
              for (int p = 0; p < PASSES; ++p) {
                uint4 x = *at(p);
                if (drop_nonfinite<PBF>(x)) {
                  *at(p) = x;
                  const int j = j0 + lw * 32 + p * RPI + lane / CH;   // (rows that no query sees: nobody asks)
                  bad |= j < it.end() && (j >= it.lo || j < it.sk);
                }
              }
              if (bad) *v_flag = 1;
              fence_async_smem();
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[k.s]);
        }
        return true;
      });
    } else {
      // ---- e4m3 pages: this warp's 32 rows of every tile of its plane. LPR lanes of 16 codes per row, RP rows a
      // pass, PN passes; the lanes of a row's second 64 columns take their two 8-code halves in the other order, so
      // that no store conflicts. Rows that no query sees are zeros. A plane's warps agree on the tile's exponent
      // bound through shared memory.
      const int plane = warp < 14 ? 0 : 1;
      constexpr int LPR = HD / 16, RP = 32 / LPR, PN = 32 / RP;
      const int ci = lane % LPR, sw = HD == 128 && ci >= 4 ? 1 : 0;
      const int c0 = ((2 * ci) & 7) + sw, c1 = ((2 * ci) & 7) + 1 - sw;
      const int mask = (1 << pg.shift) - 1;
      volatile int* bounds = (volatile int*)(sm + L::BASE) + BASES + 8 * plane;   // [2][4 warps] by tile parity
      int tiles = 0;                                             // before the item
      bool ok = true;                                            // (a warp that gave up still meets the others of its plane)
      each_item([&](const Item& it, int k, int t0, int t1) {
        if (!pair && k > 0 && ok) ok = wwait(kv_free, (k - 1) & 1);
        const int n = it.n;
        auto vector_of = [&](int t) -> int64_t {                 // of row `lane` of tile t; -1: none that a query sees
          if (t >= n) return -1;
          const int key = it.tile(t) + lw * 32 + lane;
          if (key >= it.end() || (key < it.lo && key >= it.sk)) return -1;
          const int id = pg.table[(int64_t)it.seq * pg.table_stride + (key >> pg.shift)];
          if (id < 0 || id >= pg.n_pages) return -1;
          return ((((int64_t)plane * pg.n_pages + id) * pg.Hkv + it.g) << pg.shift) + (key & mask);
        };
        uint4 code[PN];                                          // of this warp's rows of the next tile
        float sc = 0.f;                                          // and the scale of its row `lane`
        int run = NO_BOUND;
        auto read = [&](int64_t v, int p) {
          const int64_t w = __shfl_sync(0xffffffffu, v, p * RP + lane / LPR);
          return w >= 0 ? __ldg(reinterpret_cast<const uint4*>((const uint8_t*)pg.data + w * HD) + ci)
                        : make_uint4(0, 0, 0, 0);
        };
        auto fetch = [&](int64_t v) {
          sc = v >= 0 ? __ldg(pg.scales + v) : 0.f;
#pragma unroll
          for (int p = 0; p < PN; ++p) code[p] = read(v, p);
        };
        int64_t vec = vector_of(0), next = vector_of(1);         // (page ids a tile ahead of the codes)
        if (n > 0) fetch(vec);
        for (int t = 0; t < n; ++t) {
          const Slot ks = slot(t, plane == 1, t0, t1);
          // the exponent bound: K's of the tile, V's running
          const int mine = __reduce_max_sync(0xffffffffu, bound_of(sc));
          if (lane == 0) bounds[4 * ((tiles + t) & 1) + lw] = mine;
          plane_sync(plane);
          const volatile int* w4 = bounds + 4 * ((tiles + t) & 1);
          const int top = max(max(w4[0], w4[1]), max(w4[2], w4[3]));
          run = plane ? max(run, top) : top;
          const int E = run == NO_BOUND ? 0 : run;
          const int up = (7 - E) >> 1;                           // (2^(7 - E) itself may pass fp32's range)
          const float fac = sc * pow2f(up) * pow2f(7 - E - up);  // below 2^7
          if (ok) ok = wwait(&empty[ks.s], ks.ph ^ 1);
          if (!ok) continue;
          uint8_t* dst = kvst + ks.s * L::TILE;
          const bool fast = __all_sync(0xffffffffu, __half2float(__float2half_rn(fac)) == fac);
          const bool check = plane && it.partly(it.tile(t), a.window, a.sinks);
          uint8_t* d = dst + (ci >> 2) * (BKV * 128) + (lw * 32 + lane / LPR) * 128;
          bool bad = false;
          auto convert = [&](auto is_fast, const uint4 cc, int p) {
            constexpr bool FAST = decltype(is_fast)::value;
            const float f = __shfl_sync(0xffffffffu, fac, p * RP + lane / LPR);
            const int x = (p * RP + lane / LPR) & 7;
            const uint2 lo = make_uint2(cc.x, cc.y), hi = make_uint2(cc.z, cc.w);
            uint4 h0 = codes_to_half<FAST>(sw ? hi : lo, f), h1 = codes_to_half<FAST>(sw ? lo : hi, f);
            if (check) bad |= drop_nonfinite<false>(h0) | drop_nonfinite<false>(h1);
            *reinterpret_cast<uint4*>(d + p * RP * 128 + ((c0 ^ x) << 4)) = h0;
            *reinterpret_cast<uint4*>(d + p * RP * 128 + ((c1 ^ x) << 4)) = h1;
          };
          if (fast) {
#pragma unroll
            for (int p = 0; p < PN; ++p) convert(std::true_type{}, code[p], p);
          } else {                               // (rare: reads the codes again, one pass at a time)
#pragma unroll 1
            for (int p = 0; p < PN; ++p) convert(std::false_type{}, read(vec, p), p);
          }
          if (bad) *v_flag = 1;
          if (lw == 0 && lane == 0) (plane ? base_v : base_k)[(tiles + t) % BASES] = E;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(plane ? &vfull[ks.s] : &full[ks.s]);
          vec = next;
          next = vector_of(t + 2);
          if (t + 1 < n) fetch(vec);
        }
        tiles += n;
        return true;
      });
    }
  } else {
    // ---- softmax of stream x: row r = TMEM lane r
    const int x = (warp - 2) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane, r_row = r / pl.G, r_head = r % pl.G;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * 128, tO = tmem + lane_off + T_O + x * 128;
    float* qsc = (float*)(sm + L::QSC) + (pair && x ? BQ : 0);
    float* pub = reinterpret_cast<float*>(kvst) + r * L::OSTR;
    int tiles = 0, dn0 = 0, dn1 = 0;           // before the item: key tiles, and o_done phases of the two streams
    wait_prerequisites();
    each_item([&](const Item& it, int k, int t0, int t1) {
      const int n = it.n, before = x ? t1 : t0;
      struct Row {
        bool live, idle;       // idle: the warp's 32 matrix rows are past the tile's last; it only keeps the barriers going
        int pos, lo;           // position and the window's first key
        int64_t at;            // (row of q and out) * Hq + q head
      };
      auto row_of = [&](const Item& i) {
        Row w;
        const int q0 = i.v0 + (pair && x ? pl.RT : 0);     // the tile's first row of the sequence
        const int vq = q0 + r_row;                         // this row's
        w.live = r < pl.RT * pl.G && vq < i.v1 && vq < q0 + pl.RT;
        w.idle = quad * 32 >= (min(i.v1, q0 + pl.RT) - q0) * pl.G;
        w.at = ((int64_t)i.row0 + vq) * a.Hq + i.g * pl.G + r_head;
        w.pos = w.live ? i.pos0 + vq : i.end() - 1;        // (rows that are not there: any, nothing reads them)
        w.lo = a.window && w.pos - (a.window - 1) > 0 ? w.pos - (a.window - 1) : 0;
        return w;
      };
      Row rw = row_of(it);
      const bool idle = rw.idle, none = pair && x && !it.two;   // none: no second tile at all
      const int pos = rw.pos, row_lo = rw.lo;
      float sl2 = a.scale * 1.4426950408889634f;
      if constexpr (!QTMA) {   // bf16 Q rows of the quadrant to f16 (one tile: each stream half of them); absent rows are zeros
        constexpr int CH = HD / 8;
        if (!wwait(q_empty, (k & 1) ^ 1)) return false;
        const int64_t off = rw.live ? ((int64_t)it.row0 + it.v0 + (pair && x ? pl.RT : 0) + r_row) * a.q_stride +
                                          (int64_t)(it.g * pl.G + r_head) * HD : -1;
        uint8_t* dst = sm + L::Q + (pair && x ? BQ * HD * 2 : 0);
        const int first = pair ? 0 : x * (CH / 2), count = pair ? CH : CH / 2;
#pragma unroll 2
        for (int p = first; p < first + count; ++p) {      // 32 rows x CH chunks
          const int e = p * 32 + lane, rr = quad * 32 + e / CH, c = e % CH;
          const int64_t o = __shfl_sync(0xffffffffu, off, e / CH);
          const uint4 v = o >= 0 ? __ldg(reinterpret_cast<const uint4*>((const uint16_t*)a.q + o) + c)
                                 : make_uint4(0, 0, 0, 0);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t top = 0;                                // the row's largest element near 2^14
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
#pragma unroll
          for (int s = CH / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
          const int E = min(max((int)(top >> 7) - 127, -100), 127);
          const float up = __uint_as_float((uint32_t)(14 - E + 127) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = h2u(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
          if (c == 0) qsc[rr] = __uint_as_float((uint32_t)(E - 14 + 127) << 23);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (BQ * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        if (!wwait(q_full, k & 1)) return false;           // (the two streams may have loaded half of the rows each)
        sl2 *= qsc[r];
      }
      float m = -INFINITY;                       // the row's base
      uint64_t l2 = 0;                           // the row's sum, two partial sums
      int li = 0;                                // half tiles this stream has taken
      int unit = 0;                              // e4m3: O counts 2^(unit - 7)
      for (int t = pair ? 0 : x; t < n && !none; t += (li & 1) ? 0 : pair ? 1 : 2) {
        const int hh = li & 1, ph = (before + (li >> 1)) & 1;
        if (!wwait(&s_full[2 * x + hh], ph)) return false;
        ++li;
        if (idle) {
          if (lane == 0) mbar_arrive(&p_full[2 * x + hh]);
          continue;
        }
        fence_after();
        uint32_t u[64];
        tld32(tS + hh * 64, u);
        tld32(tS + hh * 64 + 32, u + 32);
        // visible keys of this half: columns lo .. hi, and those below sk
        const int base_j = it.tile(t) + hh * 64;
        const int lo = row_lo - base_j, hi = pos - base_j, sk = a.sinks - base_j;
        float zs = sl2;
        int unit_now = unit;
        if constexpr (E4) {
          // a factor that vanishes would make -inf x 0 of the hidden keys (scores are below 2^39 of it, so 0 all the same), and
          // one past fp32's range 0 x inf of a score of 0
          zs = fminf(fmaxf(zs * pow2f(base_k[(tiles + t) % BASES] - 7), 1.17549435e-38f), 3.402823466e38f);
          const Slot vs = slot(t, true, t0, t1);               // (V's bound comes with the V tile)
          if (hh == 0 && !wwait(&vfull[vs.s], vs.kind_ph)) return false;
          unit_now = base_v[(tiles + t) % BASES];
        }
        ld_wait();
        pin32(u);
        pin32(u + 32);
        // some row does not see all keys: -inf for the hidden
        if (!__all_sync(0xffffffffu, (lo <= 0 || sk >= 64) && hi >= 63)) {
          auto upto = [](int c) { return c <= 0 ? 0ull : c >= 64 ? ~0ull : ~0ull >> (64 - c); };   // columns below c
          const uint64_t seen = upto(hi + 1) & (~upto(lo) | upto(sk));
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (!((e < 32 ? (uint32_t)seen : (uint32_t)(seen >> 32)) & (1u << (e & 31)))) u[e] = 0xff800000u;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k8 = 0; k8 < 64; k8 += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx4[e] = fmaxf(mx4[e], fmaxf(__uint_as_float(u[k8 + e]), __uint_as_float(u[k8 + 4 + e])));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * zs;
        float alpha = 1.f;
        if (mx - m > TOP) {
          const float to = fabsf(mx) < FAR ? mx - HEAD : mx;
          alpha = m == -INFINITY ? 1.f : ex2(m - to);
          m = to;
        }
        const float base = m == -INFINITY ? 0.f : m;
        const bool moved = E4 && unit_now != unit;
        if (li > 1 && (moved || __any_sync(0xffffffffu, alpha != 1.f))) {   // once the last P V has completed
          if (!wwait(&o_step[2 * x + (hh ^ 1)], (before + ((li - 2) >> 1)) & 1)) return false;
          fence_after();
          const float beta = moved ? alpha * pow2f(unit - unit_now) : alpha;
          uint32_t w[16];
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            tld16(tO + c, w);
            ld_wait();
            pin<16>(w);
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * beta);
            tst16(tO + c, w);
          }
          l2 = mul2(l2, pack2(alpha, alpha));
        }
        unit = unit_now;
        const uint64_t nb = pack2(-base, -base), zs2 = pack2(zs, zs);
        uint64_t sum2 = 0;                       // (of this half: one by one, small weights would not reach a large sum)
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t z = fma2(pack2u(u[c + e], u[c + e + 1]), zs2, nb);
            const float p0 = ex2(lo2(z)), p1 = ex2(hi2(z));
            sum2 = add2(sum2, pack2(p0, p1));
            pk[e / 2] = pack_w<PBF>(p0, p1);
          }
          tst16(tS + hh * 64 + c / 2, pk);
        }
        l2 = add2(l2, sum2);
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + hh]);
      }
      // ---- the item's end (what the loop did not need is made again: registers). Its sums stay in TMEM until the
      // next item's first weights are announced
      const Item ie = item_at(k);
      rw = row_of(ie);
      float l = lo2(l2) + hi2(l2);
      if (li > 0 && !wwait(&o_done[x], (x ? dn1 : dn0) & 1)) return false;
      fence_after();
      const float scale_o = E4 ? pow2f(unit - 7) : 1.f, mean = E4 ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      float w0 = 1.f, w1 = 0.f;                  // weights of the two streams' sums
      const bool publish = !pair && x == 1;      // (o, m, l) into the K/V stages, for stream 0
      if (publish) {                             // once stream 0 has read its last tile, and the item before's sums, from them
        if (n > 0 && !wwait(&o_done[0], dn0 & 1)) return false;
        if (k > 0 && !wwait(kv_free, (k - 1) & 1)) return false;
      } else if (!pair) {
        if (!wwait(&joined[quad], k & 1)) return false;
        if (!idle) {
          const float2 ml = *reinterpret_cast<const float2*>(pub + HD);
          const bool has0 = !(m == -INFINITY && l == 0.f), has1 = !(ml.x == -INFINITY && ml.y == 0.f);
          const float M = fmaxf(m, ml.x);
          w0 = has0 ? ex2(m - M) : 0.f;
          w1 = has1 ? ex2(ml.x - M) : 0.f;
          if (m == ml.x) w0 = has0 ? 1.f : 0.f, w1 = has1 ? 1.f : 0.f;   // (also both infinite)
          const float l0 = has0 ? w0 * l : 0.f, l1 = has1 ? w1 * ml.y : 0.f;
          l = l0 + l1;
          m = M;
          if constexpr (E4) {                    // of the means
            const float one = l == 0.f ? 0.f : 1.f / l;
            w0 = l0 * one;
            w1 = l1 * one;
          }
        }
      }
      if (!idle && !none) {
        const float inv = E4 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const bool fix = rw.live && !publish && *v_flag;   // non-finite values: into the rows that see them
        const int64_t pi = (int64_t)ie.w * 2 + (pair ? x : 0);
        constexpr int CW = E4 ? 16 : 32, PIECES = CW / 8;   // columns at a time (e4m3: 96 registers a thread)
        int64_t to[PIECES];                      // where the rows of this lane's group of PIECES go
#pragma unroll
        for (int e = 0; e < PIECES; ++e) to[e] = __shfl_sync(0xffffffffu, rw.live ? rw.at : -1, (lane & ~(PIECES - 1)) + e);
#pragma unroll 1
        for (int c = 0; c < HD; c += CW) {       // (zeros without a tile)
          uint32_t u[CW];
          if (li > 0) {
            if constexpr (CW == 32) tld32(tO + c, u);
            else tld16(tO + c, u);
            ld_wait();
            pin<CW>(u);
            if constexpr (E4)
#pragma unroll
              for (int e = 0; e < CW; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * mean * scale_o);
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e) u[e] = 0u;
          }
          float4* at = reinterpret_cast<float4*>(pub + c);
          if (publish) {
#pragma unroll
            for (int e = 0; e < CW; e += 4)
              at[e / 4] = make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]), __uint_as_float(u[e + 2]),
                                      __uint_as_float(u[e + 3]));
            continue;
          }
          if (!pair) {
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
              const float4 y = at[e / 4];
              const float y4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int z = 0; z < 4; ++z)
                u[e + z] = __float_as_uint((w0 != 0.f ? w0 * __uint_as_float(u[e + z]) : 0.f) +
                                           (w1 != 0.f ? w1 * y4[z] : 0.f));
            }
          }
          if (fix) add_nonfinite<E4, PBF, CW>(ie, a, rw.pos, rw.lo, c, u);
          if (ie.ns == 1) {
            // 16-byte pieces change places within PIECES lanes, so that each store has PIECES * 16 bytes of a row
            // side by side (a row's own piece in every lane: 32 lines a store, the end of an item 3.3 us instead of
            // 2)
            uint32_t y[CW / 2];
#pragma unroll
            for (int e = 0; e < CW / 2; ++e)
              y[e] = pack_w<OBF>(__uint_as_float(u[2 * e]) * inv, __uint_as_float(u[2 * e + 1]) * inv);
#pragma unroll
            for (int step = 1; step < PIECES; step <<= 1) {
              const bool up = lane & step;
#pragma unroll
              for (int e = 0; e < PIECES; ++e)
                if (!(e & step)) {
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    uint32_t &lo_ = y[4 * e + z], &hi_ = y[4 * (e + step) + z];
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo_ : hi_, step);
                    if (up) lo_ = got;
                    else hi_ = got;
                  }
                }
            }
#pragma unroll
            for (int e = 0; e < PIECES; ++e)
              if (to[e] >= 0)
                *reinterpret_cast<uint4*>((uint16_t*)a.out + to[e] * HD + c + (lane & (PIECES - 1)) * 8) =
                    make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          } else {                               // [HD / 4][32 rows] groups of 4 sums
            float4* dst = reinterpret_cast<float4*>(a.ws) + ((pi * 4 + quad) * (HD / 4) + c / 4) * 32 + lane;
#pragma unroll
            for (int e = 0; e < CW; e += 4)
              dst[e / 4 * 32] = make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]), __uint_as_float(u[e + 2]),
                                            __uint_as_float(u[e + 3]));
          }
        }
        if (publish) *reinterpret_cast<float2*>(pub + HD) = make_float2(m, l);
        else if (rw.live && ie.ns > 1)
          reinterpret_cast<float2*>((float*)a.ws + (int64_t)tab.split * 2 * BQ * HD)[pi * BQ + r] =
              E4 ? leveled(m, l) : make_float2(m, l);
      }
      if (publish) {
        fence_async_smem();                      // (TMA tiles follow these writes)
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[quad]);
      }
      if (!pair && x == 0) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_free);
      }
      fence_before();                            // (the reads of O come before the next item's products)
      tiles += n;
      dn0 += n > 0;
      dn1 += pair ? n > 0 && it.two : n > 1;
      return true;
    });
  }
  __syncthreads();
  if ((warp == 0 || warp == 15) && *abort_flag) {   // nothing in flight when the CTA leaves
    if (q_done) mbar_drain(q_full, (q_done - 1) & 1);
    for (int s = 0; s < NS; ++s)
      if ((done >> s) & 1) mbar_drain(warp ? &vfull[s] : &full[s], (done >> (16 + s)) & 1);
  }
  if (warp == 1) {
    fence_after();
    tmem_free<TMEM_COLS>(tmem);
  }
}

// Joins the parts of a row, m their bases: M = max m, o = sum 2^(m - M) o / sum 2^(m - M) l. A part without a visible
// key (m = -inf, l = 0) holds no sums. MEANS: o / l instead of o (SHARE). A block joins 32 rows x 8 columns; warp w
// takes the parts w, w + W, ..., and the W sums are joined through shared memory: every order is fixed by the sizes.
// A warp's reads are issued together.
constexpr int CWARPS = 8, CCOLS = 8;
__device__ __forceinline__ float part_weight(float m, float M) { return m == M ? 1.f : t5::ex2(m - M); }
template <int HD, bool OBF, bool MEANS, int N>
__global__ void __launch_bounds__(CWARPS * 32, 4)
    combine_kernel(const __grid_constant__ Tab<N> tab, const __grid_constant__ PagedAttnArgs a, const Plan pl) {
  __shared__ float4 po[CWARPS][CCOLS / 4][36];
  __shared__ float2 pml[CWARPS][32];
  allow_dependents();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5, Hkv = a.pages.Hkv;
  const int cb = blockIdx.x % (HD / CCOLS), quad = blockIdx.x / (HD / CCOLS) % 4, tile = blockIdx.x / (HD / CCOLS * 4);
  int si = 0;
  while (tab.tiles[si + 1] <= tile) ++si;
  const int len = tab.len[si], ns = tab.ns[si], MT = (len + pl.RT - 1) / pl.RT, MP = (MT + pl.nt - 1) / pl.nt;
  const int lt = tile - tab.tiles[si], mt = lt % MT, g = lt / MT;
  const int rows = min(pl.RT, len - mt * pl.RT) * pl.G;        // of this query tile
  wait_prerequisites();                                        // (every CTA: a grid's end is then the one before's, too)
  if (quad * 32 >= rows) return;
  auto out_at = [&](int r) {                                   // where matrix row r of the tile goes
    return (((int64_t)tab.row0[si] + mt * pl.RT + r / pl.G) * a.Hq + g * pl.G + r % pl.G) * HD + cb * CCOLS;
  };
  // this tile's parts, two tile slots each, MP * Hkv items apart
  const int mp = mt / pl.nt;
  const int64_t p0 = ((int64_t)tab.start[si] + (int64_t)g * MP + MP - 1 - mp) * 2 + mt % pl.nt;
  const int64_t apart = (int64_t)MP * Hkv * 2;
  const float2* ml = reinterpret_cast<const float2*>((const float*)a.ws + (int64_t)tab.split * 2 * BQ * HD) + p0 * BQ +
                     quad * 32 + lane;
  const float4* ps = reinterpret_cast<const float4*>(a.ws) + ((p0 * 4 + quad) * (HD / 4) + cb * (CCOLS / 4)) * 32 + lane;
  float m = -INFINITY, l = 0.f;
  float4 o[CCOLS / 4] = {};
  constexpr int U = 4;                                         // parts read together
  for (int p = w; p < ns; p += U * W) {
    float2 x[U];
    float4 v[U][CCOLS / 4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      x[k] = make_float2(-INFINITY, 0.f);
      if (p + k * W < ns) {
        x[k] = __ldcg(ml + (p + k * W) * apart * BQ);
#pragma unroll
        for (int c = 0; c < CCOLS / 4; ++c) v[k][c] = __ldcg(ps + ((p + k * W) * apart * HD + c) * 32);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (x[k].x == -INFINITY && x[k].y == 0.f) continue;
      const float M = fmaxf(m, x[k].x), wo = part_weight(m, M), wp = part_weight(x[k].x, M);
      m = M;
      l = wo * l + wp * x[k].y;
      const float ws = MEANS ? wp * x[k].y * SHARE : wp;
#pragma unroll
      for (int c = 0; c < CCOLS / 4; ++c) {
        o[c].x = wo * o[c].x + ws * v[k][c].x;
        o[c].y = wo * o[c].y + ws * v[k][c].y;
        o[c].z = wo * o[c].z + ws * v[k][c].z;
        o[c].w = wo * o[c].w + ws * v[k][c].w;
      }
    }
  }
  pml[w][lane] = make_float2(m, l);
#pragma unroll
  for (int c = 0; c < CCOLS / 4; ++c) po[w][c][lane] = o[c];
  __syncthreads();
  constexpr int CP = CCOLS / 2;
  for (int i = threadIdx.x; i < 32 * CP; i += blockDim.x) {    // (row, 2 columns)
    const int lr = i / CP, cp = i % CP, r = quad * 32 + lr;
    if (r >= rows) continue;
    float M = -INFINITY, sum = 0.f, y0 = 0.f, y1 = 0.f;
    for (int k = 0; k < W; ++k) M = fmaxf(M, pml[k][lr].x);
    for (int k = 0; k < W; ++k) {
      const float2 x = pml[k][lr];
      if (x.x == -INFINITY && x.y == 0.f) continue;
      const float wp = part_weight(x.x, M);
      const float2 v = reinterpret_cast<const float2*>(&po[k][cp >> 1][lr])[cp & 1];
      sum += wp * x.y;
      y0 += wp * v.x;
      y1 += wp * v.y;
    }
    const float inv = sum == 0.f ? 0.f : (MEANS ? UNSHARE : 1.f) / sum;
    *reinterpret_cast<uint32_t*>((uint16_t*)a.out + out_at(r) + cp * 2) = pack_w<OBF>(y0 * inv, y1 * inv);
  }
}

// Key tiles of the item whose rows start at v0 of a sequence at pos0.
int item_tiles(int pos0, int v0, int v1, int window, int sinks) {
  const int p_first = pos0 + v0;
  Seen s;
  s.end = pos0 + v1;
  s.lo = window && p_first - (window - 1) > 0 ? p_first - (window - 1) : 0;
  s.sk = std::min(sinks, s.lo);
  return tiles_of<BKV>(s).count();
}

// One launch: sequences s0 .. (empty ones left out) with one or two query tiles an item and, per sequence, the parts
// that an item's key tiles are split into: the choice with the least estimated time (us, measured): a key tile takes
// 1.13 us with two query tiles and 0.66 with one, an item ITEM besides and a CTA's start and end 6, the join 2.8 and
// its sums. CTAs take the items in rounds: as many as there are rounds of average ones, or an even share and a third
// of the longest where lengths differ. An item is split into parts of `per` key tiles; at most 64 parts, and parts of
// at most LONGEST tiles (the tensor cores add to one sum per output and drop what lies below its last bits).
constexpr double ITEM = 3.0;
constexpr int LONGEST = 1024;
struct Group {
  Plan pl;
  Tab<TAB_LARGE> tab;
  int next;                    // the first sequence not taken
  int max_ns;
};
int64_t most_parts(int pos0, int len) { return std::max<int64_t>(64, ((int64_t)pos0 + len) / BKV / LONGEST + 2); }
void plan_group(Group& gr, int s0, int n_seq, const int* row0, const int* len, const int* pos0, int Hq, int Hkv, int hd,
                int window, int sinks, int num_sms) {
  Plan& pl = gr.pl;
  Tab<TAB_LARGE>& t = gr.tab;
  pl.G = Hq / Hkv;
  pl.RT = BQ / pl.G;
  struct Seq {
    int s, ns;
    int64_t items[2], sum[2];    // by tiles per item
    int top[2];
  };
  static thread_local std::vector<Seq> seqs;
  seqs.clear();
  int s = s0;
  int64_t all_tiles = 0, most = 0;
  for (; s < n_seq && (int)seqs.size() < TAB_LARGE; ++s) {
    if (len[s] == 0) continue;
    const int64_t MT = ((int64_t)len[s] + pl.RT - 1) / pl.RT;
    all_tiles += MT;
    most = std::max(most, most_parts(pos0[s], len[s]));
    if (!seqs.empty() && all_tiles * Hkv * most > INT_MAX) break;   // (numbers of items and join blocks stay in 31 bits)
    Seq q{s, 1, {}, {}, {}};
    for (int k = 0; k < 2; ++k) {
      const int rows = (k + 1) * pl.RT;
      q.items[k] = ((int64_t)len[s] + rows - 1) / rows;
      for (int64_t v0 = 0; v0 < len[s]; v0 += rows) {
        const int c = item_tiles(pos0[s], (int)v0, (int)std::min<int64_t>(len[s], v0 + rows), window, sinks);
        q.sum[k] += c;
        q.top[k] = std::max(q.top[k], c);
      }
    }
    seqs.push_back(q);
  }
  gr.next = s;
  pl.nt = 1;
  gr.max_ns = 1;
  t.n = t.start[0] = t.tiles[0] = t.split = 0;
  if (seqs.empty()) return;      // (nothing but empty sequences: no tiles to share out)
  double best = -1;
  int best_per = 1;
  for (int k = 0; k < 2; ++k) {
    int longest = 0;
    for (const Seq& q : seqs) longest = std::max(longest, q.top[k]);
    const double c = k ? 1.13 : 0.66;
    int last = 0;
    const int least = (longest + LONGEST - 1) / LONGEST;
    for (int parts = least; parts == least || (parts <= 64 && parts <= longest); ++parts) {
      const int per = (longest + parts - 1) / parts;
      if (per == last) continue;
      last = per;
      double cost = 0, top = 0;
      int64_t ctas = 0, joined = 0;
      for (const Seq& q : seqs) {
        const int ns = (q.top[k] + per - 1) / per;
        const int64_t n = q.items[k] * Hkv * ns;
        ctas += n;
        if (ns > 1) joined += n;
        cost += c * (double)(q.sum[k] * Hkv) + ITEM * (double)n;
        top = std::max(top, c * ((q.top[k] + ns - 1) / ns) + ITEM);
      }
      const double rounds = (double)((ctas + num_sms - 1) / num_sms), mean = cost / (double)ctas;
      double time = 6 + (ctas <= num_sms ? top : std::max(rounds * mean, cost / num_sms + 0.33 * (top - mean)));
      if (joined) time += 2.8 + 0.00006 * (double)(joined * (k + 1) * hd);
      if (best < 0 || time < best) {
        best = time;
        best_per = per;
        pl.nt = k + 1;
      }
      if (ctas > 8ll * num_sms) break;
    }
  }
  const int k = pl.nt - 1;
  for (Seq& q : seqs) q.ns = (q.top[k] + best_per - 1) / best_per;
  std::sort(seqs.begin(), seqs.end(), [&](const Seq& x, const Seq& y) {
    if ((x.ns > 1) != (y.ns > 1)) return x.ns > 1;
    if (x.ns == 1 && x.top[k] != y.top[k]) return x.top[k] > y.top[k];
    return x.s < y.s;
  });
  t.n = (int)seqs.size();
  for (int i = 0; i < t.n; ++i) {
    const Seq& q = seqs[i];
    t.row0[i] = row0 ? row0[q.s] : 0;
    t.pos0[i] = pos0[q.s];
    t.len[i] = len[q.s];
    t.seq[i] = q.s;
    t.ns[i] = q.ns;
    t.start[i + 1] = t.start[i] + (int)(q.items[k] * Hkv * q.ns);
    t.tiles[i + 1] = t.tiles[i] + (q.ns > 1 ? (int)(q.items[0] * Hkv) : 0);
    if (q.ns > 1) t.split = t.start[i + 1];
    gr.max_ns = std::max(gr.max_ns, q.ns);
  }
}

template <int HD, int KIND, int N>
cudaError_t launch_tab(const PagedAttnArgs& a, const Tab<N>& tab, const Plan& pl, int max_ns, const CUtensorMap& map,
                       int num_sms, cudaStream_t st) {
  using L = Lay<HD>;
  CUtensorMap map_q = {};
  if (KIND != E4M3_QBF) {      // (hd, q heads, rows): a tile's rows x heads are one box
    int rows = 0;
    for (int i = 0; i < tab.n; ++i) rows = std::max(rows, tab.row0[i] + tab.len[i]);
    const uint64_t dims[3] = {(uint64_t)HD, (uint64_t)a.Hq, (uint64_t)rows};
    const uint64_t str[2] = {HD * 2, (uint64_t)a.q_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)pl.G, (uint32_t)pl.RT};
    if (!encode_tensor_map(&map_q, KIND == BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, a.q,
                           dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  CK_RET(cudaFuncSetAttribute(paged_kernel<HD, KIND, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  CK_RET(launch_pdl(paged_kernel<HD, KIND, N>, dim3((unsigned)std::min(tab.start[tab.n], num_sms)), dim3(threads_of(KIND)),
                    L::BYTES, st, tab, map, map_q, a, pl));
  if (max_ns > 1)
    CK_RET(launch_pdl(combine_kernel<HD, out_bf16(KIND), is_e4m3(KIND), N>,
                      dim3((unsigned)(tab.tiles[tab.n] * (HD / CCOLS * 4))),
                      dim3((unsigned)(32 * std::min(CWARPS, (max_ns + 1) / 2))), 0, st, tab, a, pl));
  return cudaSuccess;
}
template <int HD, int KIND>
cudaError_t launch_group(const PagedAttnArgs& a, const Group& gr, int num_sms, cudaStream_t st) {
  CUtensorMap map = {};
  if (!is_e4m3(KIND) && !pages_map(&map, a.pages, 1 << a.pages.shift)) return cudaErrorInvalidValue;
  const Tab<TAB_LARGE>& t = gr.tab;
  if (t.n > TAB_SMALL) return launch_tab<HD, KIND, TAB_LARGE>(a, t, gr.pl, gr.max_ns, map, num_sms, st);
  Tab<TAB_SMALL> u;
  u.n = t.n;
  u.split = t.split;
  std::copy(t.start, t.start + t.n + 1, u.start);
  std::copy(t.tiles, t.tiles + t.n + 1, u.tiles);
  std::copy(t.row0, t.row0 + t.n, u.row0);
  std::copy(t.pos0, t.pos0 + t.n, u.pos0);
  std::copy(t.len, t.len + t.n, u.len);
  std::copy(t.seq, t.seq + t.n, u.seq);
  std::copy(t.ns, t.ns + t.n, u.ns);
  return launch_tab<HD, KIND, TAB_SMALL>(a, u, gr.pl, gr.max_ns, map, num_sms, st);
}
template <int HD>
cudaError_t launch_kind(const PagedAttnArgs& a, const Group& gr, int num_sms, cudaStream_t st) {
  if (a.pages.format == KVF_F16) return launch_group<HD, F16>(a, gr, num_sms, st);
  if (a.pages.format == KVF_BF16) return launch_group<HD, BF16>(a, gr, num_sms, st);
  return a.bf16 ? launch_group<HD, E4M3_QBF>(a, gr, num_sms, st) : launch_group<HD, E4M3>(a, gr, num_sms, st);
}
}  // namespace pgp

bool attention_paged_fits(int len, int pos0, int Hq, int Hkv) {
  const int RT = pgp::BQ / (Hq / Hkv);
  return ((int64_t)len / RT + 1) * Hkv * pgp::most_parts(pos0, len) <= INT_MAX;
}

cudaError_t attention_paged_gave_up_word(uint64_t** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), pgp::g_given_up);
}

static int64_t group_ws_bytes(const pgp::Group& gr, int hd) { return (int64_t)gr.tab.split * 2 * pgp::BQ * (hd + 2) * 4; }

int64_t attention_paged_ws_bytes(int n_seq, const int* len, const int* pos0, int Hq, int Hkv, int hd, int window, int sinks,
                                 int num_sms) {
  int64_t need = 0;
  pgp::Group gr;
  for (int s = 0; s < n_seq; s = gr.next) {
    pgp::plan_group(gr, s, n_seq, nullptr, len, pos0, Hq, Hkv, hd, window, sinks, num_sms);
    need = std::max(need, group_ws_bytes(gr, hd));
  }
  return need;
}

cudaError_t launch_attention_paged(const PagedAttnArgs& a, int n_seq, const int* row0, const int* len, const int* pos0,
                                   int num_sms, int64_t ws_bytes, bool* too_small, cudaStream_t st) {
  pgp::Group gr;
  const PagesArgs& pg = a.pages;
  *too_small = false;
  for (int s = 0; s < n_seq; s = gr.next) {
    pgp::plan_group(gr, s, n_seq, row0, len, pos0, a.Hq, pg.Hkv, pg.hd, a.window, a.sinks, num_sms);
    if (s == 0) {              // before anything is launched: the workspace of all groups (one, mostly)
      const int64_t need = gr.next == n_seq ? group_ws_bytes(gr, pg.hd)
                                            : attention_paged_ws_bytes(n_seq, len, pos0, a.Hq, pg.Hkv, pg.hd, a.window,
                                                                       a.sinks, num_sms);
      if (need > 0 && (!a.ws || ws_bytes < need)) {
        *too_small = true;
        return cudaSuccess;
      }
    }
    if (gr.tab.n == 0) continue;
    CK_RET(pg.hd == 128 ? pgp::launch_kind<128>(a, gr, num_sms, st) : pgp::launch_kind<64>(a, gr, num_sms, st));
  }
  return cudaSuccess;
}

}  // namespace s1
