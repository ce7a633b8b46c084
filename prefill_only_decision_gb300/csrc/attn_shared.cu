// Attention of a batch of sequences over one shared prefix, on the 5th-generation tensor cores.
//
// Query row i of sequence s attends to the P rows of the snapshot and to rows 0 .. i of its own
// sequence: o = softmax(scale q.k) v. All sequences see the same prefix, so their query rows (and
// the G = Hq / Hkv q heads that share a kv head) are packed into tiles of 128 matrix rows:
// RT = floor(128 / G) query rows x G heads per tile, whichever sequences the rows belong to. A
// tile reads each 128-key tile of the prefix once; s1_op_attention's kernel, one tile per
// (sequence, q head), reads it once per sequence and head.
//
// One pass over the keys with a running base (near the maximum) and sum in fp32, in two streams of S = Q K^T,
// softmax, O += P V that share the tensor cores. The streams are two query tiles over the same key
// tiles or, with one query tile an item (small calls, and the last of an odd count), that tile over
// the even and the odd key tiles, joined at the end. A stream takes a key tile in two halves of 64
// keys with S in TMEM columns of their own: while the softmax works on one half, the products P V of
// the half before and S of the half behind it run. (One S of 128 columns: softmax and products of a
// stream take turns, and both streams' products collide; 65536 rows, 1340 packed rows x 16 heads: 574
// us, in halves 471, or 525 after a second of load, when the clock has come down. The halves' S reads Q
// twice, 1.5 x the shared-memory time of S.)
// Work items are (kv head, query tile or pair of tiles); an item's key tiles are split over `ns` CTAs
// when that shortens the call, and combine_kernel joins their (o, m, l) in an order that the sizes fix
// (no atomics: the same bits every time). One CTA per SM, 15 warps (19 with an e4m3 prefix):
//   warp 0      TMA producer: f16 prefix tiles
//   warps 1, 14 MMA issue of stream 0 and 1
//   warps 2-5, 6-9  softmax of stream 0, 1: one thread per row (TMEM lane), 64 scores in registers.
//               Running base with a lazy rescale (O and l move only when the row's weights would pass
//               2^TOP, once the last P V has completed). P (f16) goes back into the TMEM columns of
//               S and is the A operand of O += P V from there: no shared-memory round trip. Warps whose
//               32 rows are all past the tile's last row leave at once: their polling slowed the others.
//   warps 10-13 loaders: the batch's own keys (gathered row by row through the sequence table), and
//               e4m3 prefix tiles: codes from memory through registers (read one tile ahead, asked for in
//               L2 three ahead) to f16 in the MMA's swizzled layout. With an e4m3 prefix they take the K
//               tiles and warps 15-18 the V tiles. (Codes through a shared-memory ring cost a third of
//               its bandwidth, the bound of this kernel: 65536 rows 645 us, straight from memory 544.)
// K and V tiles share one ring of stages in the order the products take them. Each role is one short
// loop with one copy of its body: the roles together overflow the instruction cache when they are
// inlined several times (four copies: f16 491 us instead of 470, e4m3 571 instead of 544).
// Own keys are packed the same way as queries: row r's visible own keys are the packed rows
// start(r) .. r, so one masked tile serves many short sequences. A masked weight is an exact zero,
// but 0 x NaN is not: the loaders replace non-finite own V elements by 0 and flag the CTA, and
// the epilogue then adds them to exactly the rows that see them.
// An e4m3 code times its scale is exact in f16 for scales 2^-6 .. 2^7 (and rounded as the read-back
// rounds it otherwise), so the products run on f16 operands as with an f16 snapshot.
// Every mbarrier wait is bounded; on expiry an error word is set and every role leaves.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace sha {
using namespace t5;

constexpr int BQ = 128, BKV = 128;
constexpr int threads_of(bool e4m3) { return (e4m3 ? 19 : 15) * 32; }
constexpr int TMEM_COLS = 512;               // S of stream x at 128 x, O at 256 + 128 x
constexpr int T_O = 256;
// Weights are 2^(z - m), z the score (log2 domain) and m a base that a row moves to HEAD below its maximum when they
// would pass 2^TOP, within f16. So a weight keeps f16's precision down to 2^-24 of the largest, and one that is
// lost is below 2^-35 of it: 65536 of those are 2^-19 of the result. (A base at the maximum, moved when that grew by
// 2^8, lost what lies below 2^-25: behind a sink, all of the result. HEAD of 7, 9, 10, 11, 12: 1340 rows over 65536
// keys 472, 471, 473, 478, 484 us.) Maxima past FAR are their own base: fp32 does not hold HEAD beside them.
constexpr float HEAD = 10.f, TOP = 15.f, FAR = 4194304.f;

__device__ uint64_t g_given_up;              // when a bounded wait last gave up, per device; never cleared

struct Plan {
  int V;          // packed query rows
  int G, RT, MT;  // q heads per kv head, query rows per tile, tiles
  int MP;         // work items per kv head: tiles or pairs of tiles
  int nt;         // tiles per item (1 or 2; the last item of an odd count has one)
  int ns;         // key parts per item
  int ncache;     // prefix tiles
};

// Shared memory: Q tiles, then stages of f16 K or V tiles. Two query tiles: F stages that both streams
// read; one query tile: its Q and a ring of FR stages for each stream (227 KB at hd 128: 2 x 32 + 5 x 32,
// or 1 x 32 + 6 x 32).
template <int HD>
struct Lay {
  static constexpr int TILE = BKV * HD * 2;
  static constexpr int F = HD == 128 ? 5 : 7;
  static constexpr int FR = (F + 1) / 2;
  static constexpr int Q = 0;                             // per tile HD/64 boxes of [128 rows][128 B]
  static constexpr int KV2 = Q + 2 * BQ * HD * 2;         // stages with two query tiles
  static constexpr int KV1 = Q + BQ * HD * 2;             // with one
  static constexpr int TAB = KV2 + F * TILE;              // a copy of a small sequence table
  static constexpr int BAR = TAB + (2 * SEQ_TAB_SMALL + 2) * 4;
  static constexpr int NS = 2 * FR > F ? 2 * FR : F;
  static constexpr int NBAR = 1 + 2 * NS + 12 + 2 + 2 + 4;
  static constexpr int USED = BAR + NBAR * 8 + 16;
  static_assert(USED <= 227 * 1024, "shared memory of one CTA");
  // above half an SM: each CTA allocates all of TMEM, so two never share one
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr int OSTR = HD + 4;                     // floats per row of a stream's published sums
  static_assert(KV1 + 2 * FR * TILE <= TAB, "both rings fit");
  static_assert(BQ * OSTR * 4 <= 2 * FR * TILE, "published sums fit the K/V stages");
};

// A stage of the ring of K and V tiles. With two query tiles both streams read one ring K_0, V_0, K_1, ...;
// with one, each stream has its own, of its tiles: a parity wait must never run more than one phase ahead
// of a slot, which waiting past the other stream's fills (they complete in any order) could.
struct Slot {
  int s;
  uint32_t ph;
};
template <int F, int FR>
__device__ __forceinline__ Slot slot_of(bool two, int t, bool is_v) {
  const uint32_t i = 2 * (two ? t : t >> 1) + (is_v ? 1 : 0);
  if (two) return {(int)(i % F), i / F & 1};
  return {(t & 1 ? FR : 0) + (int)(i % FR), i / FR & 1};
}

// Sequence tables as a kernel searches them: a small one from its copy in shared memory, a large
// one where it is.
struct TabView {
  int n;
  const int *cum, *row0;
};
// The sequence that packed row vr (< cum[n]) belongs to.
__device__ __forceinline__ int seq_of(const TabView& t, int vr) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.cum[mid] <= vr) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool nonfinite2(uint32_t h2) {   // either f16 of the pair
  return (h2 & 0x7c00u) == 0x7c00u || (h2 & 0x7c000000u) == 0x7c000000u;
}
__device__ __forceinline__ uint32_t drop_nonfinite2(uint32_t h2) {
  if ((h2 & 0x7c00u) == 0x7c00u) h2 &= 0xffff0000u;
  if ((h2 & 0x7c000000u) == 0x7c000000u) h2 &= 0xffffu;
  return h2;
}

// Eight e4m3 codes times scale to f16 (round to nearest even, held at +-65504). FAST: the scale
// is an f16 value of at most 2^7, so the f16 product is the rounded value and cannot overflow.
template <bool FAST>
__device__ __forceinline__ uint4 codes_to_half(const uint2 c, float scale) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    __half2 y;
    if constexpr (FAST) {
      y = __hmul2(x, __float2half2_rn(scale));
    } else {
      const float2 f = __half22float2(x);
      const float a = f.x * scale, b = f.y * scale;
      y = __floats2half2_rn(fabsf(a) > 65504.f ? copysignf(65504.f, a) : a,
                            fabsf(b) > 65504.f ? copysignf(65504.f, b) : b);
    }
    h[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

template <int HD, bool E4M3, int N>
__global__ void __launch_bounds__(threads_of(E4M3), 1)
    shared_kernel(const __grid_constant__ SeqTab<N> table, const __grid_constant__ CUtensorMap mapKV,
                  const __grid_constant__ SharedAttnArgs a, const Plan pl) {
  using L = Lay<HD>;
  constexpr int NB = HD / 64, F = L::F, FR = L::FR, NS = L::NS;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = (uint64_t*)(sm + L::BAR);
  uint64_t* q_full = bars;
  uint64_t* full = bars + 1;                   // [NS]
  uint64_t* empty = full + NS;                 // [NS]
  uint64_t* s_full = empty + NS;               // [2 streams][2 halves of the key tile]
  uint64_t* p_full = s_full + 4;               // [2][2]
  uint64_t* o_step = p_full + 4;               // [2][2] the half's P V has completed
  uint64_t* o_done = o_step + 4;               // [2] the stream's last product has completed
  uint64_t* mma_idle = o_done + 2;             // [2]
  uint64_t* joined = mma_idle + 2;             // [4 quadrants] stream 1's sums are published
  uint32_t* tmem_slot = (uint32_t*)(bars + L::NBAR);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* v_flag = (volatile int*)(tmem_slot + 2);   // some own V element of this CTA is not finite

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % pl.ns), item = (int)(blockIdx.x / pl.ns);
  const int mp = item % pl.MP, g = item / pl.MP;
  const bool two = pl.nt == 2 && 2 * mp + 1 < pl.MT;         // two query tiles; else one over alternate key tiles
  const int v0 = pl.nt * mp * pl.RT;               // first packed row of the item, and one past its last
  const int v1 = min(pl.V, v0 + (two ? 2 : 1) * pl.RT);

  // quadrants of 32 matrix rows that stream x's query tile fills (a single tile: both streams')
  auto quads = [&](int x) { return (min(pl.RT, pl.V - (v0 + (two && x ? pl.RT : 0))) * pl.G + 31) / 32; };
  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], E4M3 ? 4 : 5);
      mbar_init(&empty[s], two ? 2 : 1);       // the streams that read the slot
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&mma_idle[x], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[2 * x + h], 1);
        mbar_init(&p_full[2 * x + h], quads(x));
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
  TabView tab{table.n, table.cum, table.row0};
  if constexpr (N == SEQ_TAB_SMALL) {
    int* copy = reinterpret_cast<int*>(sm + L::TAB);
    if (threadIdx.x >= 64 && threadIdx.x < 64 + N) {
      const int i = threadIdx.x - 64;
      if (i < table.n) {
        copy[i] = table.cum[i];
        copy[N + 1 + i] = table.row0[i];
      }
    }
    tab.cum = copy;
    tab.row0 = copy + N + 1;
  }
  allow_dependents();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  // key tiles of this part: prefix tiles 0 .. ncache-1, then own tiles from packed row kb on
  const int kb = a.kn ? tab.cum[seq_of(tab, v0)] : 0;
  const int nown = a.kn ? (v1 - kb + BKV - 1) / BKV : 0;
  const int total = pl.ncache + nown;
  const int per = (total + pl.ns - 1) / pl.ns;
  const int jb = min(total, part * per), je = min(total, jb + per);
  const int n = je - jb;
  uint8_t* kvst = sm + (two ? L::KV2 : L::KV1);

  if (warp == 0) {
    // ---- TMA producer: prefix tiles of an f16 snapshot
    wait_prerequisites();
    if constexpr (!E4M3) {
      if (lane == 0) {
        uint32_t fills = 0;                    // per slot: begun (bit s), parity of the last fill (bit 16 + s)
        const int lead = two ? 1 : 2;          // K_0 .. K_{lead-1}, then V_t, K_{t+lead}
        for (int q = 0; q < 2 * n + lead - 1; ++q) {
          const int e = q - lead;
          const bool is_v = e >= 0 && !(e & 1);
          const int t = e < 0 ? q : is_v ? e >> 1 : lead + (e >> 1), j = jb + t;
          if (t >= n) continue;
          const Slot k = slot_of<F, FR>(two, t, is_v);
          const int s = k.s;
          if (!mbar_wait(&empty[s], k.ph ^ 1, abort_flag, &g_given_up)) break;
          if (j < pl.ncache) {
            mbar_expect_tx(&full[s], L::TILE);
            for (int b = 0; b < NB; ++b)
              tma4(kvst + s * L::TILE + b * BKV * 128, &mapKV, &full[s], 64 * b, g, j * BKV, is_v ? 1 : 0);
          } else {
            mbar_arrive(&full[s]);
          }
          fills = (fills & ~(1u << (16 + s))) | 1u << s | k.ph << (16 + s);
        }
        if (*abort_flag)
          for (int s = 0; s < NS; ++s)
            if ((fills >> s) & 1) mbar_drain(&full[s], (fills >> (16 + s)) & 1);
      }
    }
  } else if (warp == 1 || warp == 14) {
    // ---- MMA issue of stream x: the whole warp waits, one lane issues. A stream's products run in
    // the order they are issued, so S of its next tile may take the columns that P V reads before it
    const int x = warp == 1 ? 0 : 1;
    const bool leader = elect_one();
    constexpr uint32_t ID_S = idesc_f16(BKV / 2, 0, 0, 0), ID_O = idesc_f16(HD, 0, 0, 1);
    const uint32_t tS = tmem + x * 128, tO = tmem + T_O + x * 128;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_given_up) ? 1 : 0) != 0;
    };
    const uint64_t qd = desc_sw128(smem_u32(sm + L::Q) + (two && x ? BQ * HD * 2 : 0), 16);
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
    // of each half h: P V of tile i - 1, then S of tile i into the same columns
    const int cnt = two ? n : (n + 1 - x) >> 1;
    if (cnt > 0 && wait(q_full, 0))
      for (int i = 0; i <= cnt; ++i) {
        const int t = two ? i : 2 * i + x;
        const Slot k = slot_of<F, FR>(two, t, false);                    // (unused at i = cnt)
        const Slot v = slot_of<F, FR>(two, t - (two ? 1 : 2), true);     // (unused at i = 0)
        auto half = [&](auto hc) {
          constexpr int h = decltype(hc)::value;
          if (i > 0) {
            if (h == 0 && !wait(&full[v.s], v.ph)) return false;
            if (!wait(&p_full[2 * x + h], (i - 1) & 1)) return false;
            fence_after();
            if (leader) {
              values(h, v.s, h > 0 || i > 1);
              if (h) commit(&empty[v.s]);
              if (h && i == cnt) commit(&o_done[x]);
            }
            __syncwarp();
          }
          if (i < cnt) {
            if (h == 0) {
              if (!wait(&full[k.s], k.ph)) return false;
              fence_after();
            }
            if (leader) {
              scores(h, k.s);
              if (h) commit(&empty[k.s]);
            }
            __syncwarp();
          }
          return true;
        };
        if (!half(std::integral_constant<int, 0>{}) || !half(std::integral_constant<int, 1>{})) break;
      }
    if (leader) {
      commit(&mma_idle[x]);
      mbar_drain(&mma_idle[x], 0);             // every MMA issued above has completed
    }
  } else if (warp >= 10 && warp != 14) {
    // ---- loaders: rows 32 lw .. +31 of every tile
    const int lw = warp < 14 ? warp - 10 : warp - 15, plane = warp < 14 ? 0 : 1;   // (f16 prefix: both planes)
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_given_up) ? 1 : 0) != 0;
    };
    // own rows of tile jo: CH chunks of 16 bytes per row, RPI rows per pass of the warp
    constexpr int CH = HD / 8, RPI = 32 / CH, PASSES = 32 / RPI;
    auto load_own = [&](int jo, const f16* src, uint8_t* dst, bool is_v) {
      const int kv = kb + jo * BKV + lw * 32 + lane;          // this lane's packed row
      int64_t off = -1;
      if (kv < v1) {
        const int s = seq_of(tab, kv);
        off = ((int64_t)tab.row0[s] + (kv - tab.cum[s])) * a.kv_stride + (int64_t)g * HD;
      }
      const int c = lane % CH;
      bool bad = false;
      constexpr int BATCH = E4M3 ? PASSES / 2 : PASSES;       // reads issued together (registers)
#pragma unroll 1
      for (int p0 = 0; p0 < PASSES; p0 += BATCH) {
        uint4 x[BATCH];
#pragma unroll
        for (int p = 0; p < BATCH; ++p) {
          const int64_t o = __shfl_sync(0xffffffffu, off, (p0 + p) * RPI + lane / CH);
          x[p] = o >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + o) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < BATCH; ++p) {
          if (is_v && (nonfinite2(x[p].x) || nonfinite2(x[p].y) || nonfinite2(x[p].z) || nonfinite2(x[p].w))) {
            bad = true;
            x[p] = make_uint4(drop_nonfinite2(x[p].x), drop_nonfinite2(x[p].y), drop_nonfinite2(x[p].z),
                              drop_nonfinite2(x[p].w));
          }
          const int r = lw * 32 + (p0 + p) * RPI + lane / CH;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (BKV * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x[p];
        }
      }
      if (bad) *v_flag = 1;
    };
    // e4m3 prefix: LPR lanes of 16 codes per row, RP rows a pass, PN passes; the lanes of a row's second 64
    // columns take their two 8-code halves in the other order, so that no store conflicts
    constexpr int LPR = HD / 16, RP = 32 / LPR, PN = 32 / RP;
    const int ci = lane % LPR, sw = HD == 128 && ci >= 4 ? 1 : 0;
    const int c0 = ((2 * ci) & 7) + sw, c1 = ((2 * ci) & 7) + 1 - sw;
    const int64_t krow = (int64_t)a.Hkv * HD;              // bytes from key to key
    const uint8_t* codes = (const uint8_t*)a.kv + (int64_t)plane * a.cap * krow + (int64_t)g * HD;
    const float* scales = a.scales + ((int64_t)plane * a.Hkv + g) * a.cap;
    uint4 code[PN];                                        // of this warp's rows of its plane's next tile
    float sc = 0.f;                                        // and the scale of its row `lane`
    auto read = [&](int j, int p) {                        // (rows past the prefix: codes and scales are zeros)
      const int key = j * BKV + lw * 32 + p * RP + lane / LPR;
      return key < a.P ? __ldg(reinterpret_cast<const uint4*>(codes + key * krow) + ci) : make_uint4(0, 0, 0, 0);
    };
    auto fetch_scale = [&](int j) {
      const int key = j * BKV + lw * 32 + lane;
      sc = key < a.P ? __ldg(scales + key) : 0.f;
    };
    auto prefetch = [&](int j) {
      const int key = j * BKV + lw * 32 + lane;
      if (j >= min(pl.ncache, je) || key >= a.P) return;   // (nothing behind the prefix: it may end the allocation)
      l2_prefetch(codes + key * krow);
      if (lane == 0) l2_prefetch(scales + key);
    };
    wait_prerequisites();
    if constexpr (E4M3)
      if (jb < min(pl.ncache, je)) {
        fetch_scale(jb);
#pragma unroll
        for (int p = 0; p < PN; ++p) code[p] = read(jb, p);
        prefetch(jb + 1);
        prefetch(jb + 2);
      }
    // A plane's warps see every second fill of a slot only; a parity wait needs all fills but the last to be
    // over, and they are: the warps' own last tile came after the consumption of an item behind those.
    for (int it = 0; it < (E4M3 ? n : 2 * n); ++it) {
      const int t = E4M3 ? it : it >> 1;
      const bool is_v = E4M3 ? plane == 1 : it & 1;
      const Slot k = slot_of<F, FR>(two, t, is_v);
      const int s = k.s, j = jb + t;
      if (!wwait(&empty[s], k.ph ^ 1)) break;
      uint8_t* dst = kvst + s * L::TILE;
      if (j >= pl.ncache) {
        load_own(j - pl.ncache, is_v ? a.vn : a.kn, dst, is_v);
      } else if constexpr (E4M3) {
        const bool fast = __all_sync(0xffffffffu, fabsf(sc) <= 128.f && __half2float(__float2half_rn(sc)) == sc);
        uint8_t* d = dst + (ci >> 2) * (BKV * 128) + (lw * 32 + lane / LPR) * 128;
        const bool more = j + 1 < min(pl.ncache, je);
        const float rsc = sc;
        auto convert = [&](auto is_fast, const uint4 cc, int p) {
          constexpr bool FAST = decltype(is_fast)::value;
          const float rs = __shfl_sync(0xffffffffu, rsc, p * RP + lane / LPR);
          const int x = (p * RP + lane / LPR) & 7;
          const uint2 lo = make_uint2(cc.x, cc.y), hi = make_uint2(cc.z, cc.w);
          *reinterpret_cast<uint4*>(d + p * RP * 128 + ((c0 ^ x) << 4)) = codes_to_half<FAST>(sw ? hi : lo, rs);
          *reinterpret_cast<uint4*>(d + p * RP * 128 + ((c1 ^ x) << 4)) = codes_to_half<FAST>(sw ? lo : hi, rs);
        };
        if (fast) {
#pragma unroll
          for (int p = 0; p < PN; ++p) convert(std::true_type{}, code[p], p);
        } else {                               // (rare: reads the codes again, one pass at a time)
#pragma unroll 1
          for (int p = 0; p < PN; ++p) convert(std::false_type{}, read(j, p), p);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        prefetch(j + 3);
        if (more) {                            // (behind the fence, which waits for reads in flight too)
          fetch_scale(j + 1);
#pragma unroll
          for (int p = 0; p < PN; ++p) code[p] = read(j + 1, p);
        }
        continue;
      }
      fence_async_smem();                          // this warp's writes are the MMA's to read (the producer's
      __syncwarp();                                // tiles: only the arrival)
      if (lane == 0) mbar_arrive(&full[s]);
    }
  } else {
    // ---- softmax of stream x: row r = TMEM lane r
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_given_up) ? 1 : 0) != 0;
    };
    const int x = (warp - 2) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const int q0 = v0 + (two && x ? pl.RT : 0);          // the tile's first packed row
    const int vq = q0 + r / pl.G;                        // this row's
    const bool live = r < pl.RT * pl.G && vq < v1 && vq < q0 + pl.RT;
    const int h = g * pl.G + r % pl.G;
    int vs = 0;
    int64_t row = -1;                                    // row of q and out
    if (live) {
      const int s = seq_of(tab, vq);
      vs = tab.cum[s];
      row = (int64_t)tab.row0[s] + (vq - vs);
    }
    const bool idle = quad >= quads(x);                  // no live row: nothing to do past Q's zeros
    wait_prerequisites();
    {   // Q rows of the quadrant; absent rows are zeros. One tile: each stream loads half of the chunks
      constexpr int CH = HD / 8;
      const int64_t off = live ? row * a.q_stride + (int64_t)h * HD : -1;
      uint8_t* dst = sm + L::Q + (two && x ? BQ * HD * 2 : 0);
      auto load = [&](auto count, int first) {           // `count` of the CH passes over 32 rows x CH chunks
        constexpr int PN = decltype(count)::value;
        uint4 v[PN];
#pragma unroll
        for (int p = 0; p < PN; ++p) {
          const int e = (first + p) * 32 + lane;
          const int64_t o = __shfl_sync(0xffffffffu, off, e / CH);
          v[p] = o >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + o) + e % CH) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < PN; ++p) {
          const int e = (first + p) * 32 + lane, rr = quad * 32 + e / CH, c = e % CH;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (BQ * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v[p];
        }
      };
      if (two) load(std::integral_constant<int, CH>{}, 0);
      else load(std::integral_constant<int, CH / 2>{}, x * (CH / 2));
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * 128, tO = tmem + lane_off + T_O + x * 128;
    const float sl2 = a.scale * 1.4426950408889634f;
    const uint64_t sl2_2 = pack2(sl2, sl2);
    float m = -INFINITY;                       // the row's base
    uint64_t l2 = 0;                           // the row's sum, two partial sums
    bool ok = true;
    int li = 0;                                // half tiles this stream has taken
    for (int t = two ? 0 : x; t < n && ok && !idle; t += (li & 1) ? 0 : two ? 1 : 2) {
      const int hh = li & 1, ph = (li >> 1) & 1;
      if (!wwait(&s_full[2 * x + hh], ph)) { ok = false; break; }
      ++li;
      fence_after();
      uint32_t u[64];
      tld32(tS + hh * 64, u);
      tld32(tS + hh * 64 + 32, u + 32);
      // visible keys of this half: columns lo .. hi
      const int j = jb + t;
      int lo = 0, hi;
      if (j < pl.ncache) {
        hi = a.P - 1 - j * BKV - hh * 64;
      } else {
        const int base = kb + (j - pl.ncache) * BKV + hh * 64;
        lo = vs - base;
        hi = live ? vq - base : -1;
      }
      ld_wait();
      pin32(u);
      pin32(u + 32);
      if (!__all_sync(0xffffffffu, lo <= 0 && hi >= 63)) {   // some row does not see all keys: -inf for the hidden
        const int a0 = min(max(lo, 0), 64), a1 = min(max(hi + 1, 0), 64);   // columns a0 .. a1-1
        const uint64_t seen = a1 > a0 ? (~0ull >> (64 - (a1 - a0))) << a0 : 0ull;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (!((e < 32 ? (uint32_t)seen : (uint32_t)(seen >> 32)) & (1u << (e & 31)))) u[e] = 0xff800000u;
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 64; k += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mx4[e] = fmaxf(mx4[e], fmaxf(__uint_as_float(u[k + e]), __uint_as_float(u[k + 4 + e])));
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
      float alpha = 1.f;
      if (mx - m > TOP) {
        const float to = fabsf(mx) < FAR ? mx - HEAD : mx;
        alpha = m == -INFINITY ? 1.f : ex2(m - to);
        m = to;
      }
      const float base = m == -INFINITY ? 0.f : m;
      if (li > 1 && __any_sync(0xffffffffu, alpha != 1.f)) {   // once the last P V has completed
        if (!wwait(&o_step[2 * x + (hh ^ 1)], ((li - 2) >> 1) & 1)) { ok = false; break; }
        fence_after();
        uint32_t w[16];
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          tld16(tO + c, w);
          ld_wait();
          pin<16>(w);
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
          tst16(tO + c, w);
        }
        l2 = mul2(l2, pack2(alpha, alpha));
      }
      const uint64_t nb = pack2(-base, -base);
      uint64_t sum2 = 0;                       // (of this half: one by one, small weights would not reach a large sum)
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t z = fma2(pack2u(u[c + e], u[c + e + 1]), sl2_2, nb);
          const float p0 = ex2(lo2(z)), p1 = ex2(hi2(z));
          sum2 = add2(sum2, pack2(p0, p1));
          pk[e / 2] = h2u(p0, p1);
        }
        tst16(tS + hh * 64 + c / 2, pk);
      }
      l2 = add2(l2, sum2);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * x + hh]);
    }
    // ---- epilogue
    float l = lo2(l2) + hi2(l2);
    if (ok && li > 0) ok = wwait(&o_done[x], 0);
    fence_after();
    auto sums = [&](int c, float* o) {         // 32 columns of this row's sums (zeros without a tile)
      uint32_t w[32];
      __syncwarp();
      if (li > 0) {
        tld32(tO + c, w);
        ld_wait();
        pin32(w);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = li > 0 ? __uint_as_float(w[e]) : 0.f;
    };
    float* pub = reinterpret_cast<float*>(kvst) + r * L::OSTR;
    float w0 = 1.f, w1 = 0.f;                  // weights of the two streams' sums
    if (!two && x == 1 && !idle) {
      // publish (o, m, l) in the K/V stages once stream 0 has read its last tile from them
      if (ok && n > 0) ok = wwait(&o_done[0], 0);
      if (ok) {
        float o[32];
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          sums(c, o);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(pub + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        *reinterpret_cast<float2*>(pub + HD) = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[quad]);
      }
    } else if (!idle) {
      if (!two && ok) {
        ok = wwait(&joined[quad], 0);
        if (ok) {
          const float2 ml = *reinterpret_cast<const float2*>(pub + HD);
          const bool has0 = !(m == -INFINITY && l == 0.f), has1 = !(ml.x == -INFINITY && ml.y == 0.f);
          const float M = fmaxf(m, ml.x);
          w0 = has0 ? ex2(m - M) : 0.f;
          w1 = has1 ? ex2(ml.x - M) : 0.f;
          if (m == ml.x) w0 = has0 ? 1.f : 0.f, w1 = has1 ? 1.f : 0.f;   // (also both infinite)
          l = (has0 ? w0 * l : 0.f) + (has1 ? w1 * ml.y : 0.f);
          m = M;
        }
      }
      if (ok) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool fix = live && *v_flag;      // non-finite own V elements: into the rows that see them
        const int k0 = max(vs, kb + (max(jb, pl.ncache) - pl.ncache) * BKV);
        const int k1 = min(vq, kb + (je - pl.ncache) * BKV - 1);
        const int64_t pi = (int64_t)blockIdx.x * pl.nt + (two ? x : 0);
        uint8_t* ostage = sm + L::Q + (two && x ? BQ * HD * 2 : 0);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          sums(c, o);
          if (!two) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = *reinterpret_cast<const float4*>(pub + c + e);
              o[e] = (w0 != 0.f ? w0 * o[e] : 0.f) + (w1 != 0.f ? w1 * y.x : 0.f);
              o[e + 1] = (w0 != 0.f ? w0 * o[e + 1] : 0.f) + (w1 != 0.f ? w1 * y.y : 0.f);
              o[e + 2] = (w0 != 0.f ? w0 * o[e + 2] : 0.f) + (w1 != 0.f ? w1 * y.z : 0.f);
              o[e + 3] = (w0 != 0.f ? w0 * o[e + 3] : 0.f) + (w1 != 0.f ? w1 * y.w : 0.f);
            }
          }
          if (fix)                             // (a row that is not live has no own rows)
            for (int kv = k0; kv <= k1; ++kv) {
              const f16* vp = a.vn + (row - (vq - kv)) * a.kv_stride + (int64_t)g * HD + c;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = h2f(vp[e]);
                if (!isfinite(y)) o[e] += y;
              }
            }
          if (pl.ns == 1) {                    // f16 row into the (consumed) Q tile, chunks swizzled
            uint8_t* dst = ostage + r * (HD * 2);
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + ((((c + e) / 8) ^ (r & 7)) << 4)) =
                  make_uint4(h2u(o[e] * inv, o[e + 1] * inv), h2u(o[e + 2] * inv, o[e + 3] * inv),
                             h2u(o[e + 4] * inv, o[e + 5] * inv), h2u(o[e + 6] * inv, o[e + 7] * inv));
          } else {                             // the warp's [HD / 8][32] groups of 4 sums, half of the columns at a time
            float4* stage = reinterpret_cast<float4*>(ostage + quad * (HD * 64));
            const int half = HD / 2, cc = c % half;
            if (c == half) {                   // the first half is out of the stage
              if (lane == 0) tma_store_read_wait();
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              stage[(cc + e) / 4 * 32 + lane] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            if (cc + 32 == half) {
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                bulk_store((float*)a.ws + ((pi * 4 + quad) * HD + c + 32 - half) * 32, stage, HD * 64);
                tma_store_commit();
              }
            }
          }
        }
        if (pl.ns == 1) {                      // whole rows out of the warp's stage
          __syncwarp();
          constexpr int CH = HD / 8;
          const int64_t off = live ? (row * a.Hq + h) * HD : -1;
#pragma unroll
          for (int p = 0; p < CH; ++p) {
            const int e = p * 32 + lane, rr = quad * 32 + e / CH, c = e % CH;
            const int64_t o = __shfl_sync(0xffffffffu, off, e / CH);
            if (o >= 0)
              *reinterpret_cast<uint4*>(a.out + o + c * 8) =
                  *reinterpret_cast<const uint4*>(ostage + rr * (HD * 2) + ((c ^ (rr & 7)) << 4));
          }
        }
        if (pl.ns > 1 && lane == 0) tma_store_wait();
        if (live && pl.ns > 1)
          reinterpret_cast<float2*>((float*)a.ws + (int64_t)gridDim.x * pl.nt * BQ * HD)[pi * BQ + r] = make_float2(m, l);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<TMEM_COLS>(tmem);
  }
}

// Joins the parts of a row, m their bases: M = max m, o = sum 2^(m - M) o / sum 2^(m - M) l. A part without a
// visible key (m = -inf, l = 0) holds no sums. A block joins 32 rows x 8 columns; warp w takes the parts w, w + W, ...,
// and the W sums are joined through shared memory: every order is fixed by the sizes. All of a warp's reads
// are issued together (reading m before o, part after part, cost 5.6 us for 9 parts and 9 us for 19, mostly
// round trips to L2).
constexpr int CWARPS = 8, CCOLS = 8;
__device__ __forceinline__ float part_weight(float m, float M) { return m == M ? 1.f : t5::ex2(m - M); }
template <int HD, int N>
__global__ void __launch_bounds__(CWARPS * 32, 4)
    combine_kernel(const __grid_constant__ SeqTab<N> table, const __grid_constant__ SharedAttnArgs a, const Plan pl) {
  __shared__ float4 po[CWARPS][CCOLS / 4][36];
  __shared__ float2 pml[CWARPS][32];
  allow_dependents();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5;
  const int cb = blockIdx.x % (HD / CCOLS), quad = blockIdx.x / (HD / CCOLS) % 4, tile = blockIdx.x / (HD / CCOLS * 4);
  const int mt = tile % pl.MT, g = tile / pl.MT;
  const int rows = min(pl.RT, pl.V - mt * pl.RT) * pl.G;       // of this query tile
  if (quad * 32 >= rows) {
    wait_prerequisites();                                      // (every CTA: a grid's end is then the one before's, too)
    return;
  }
  const TabView tab{table.n, table.cum, table.row0};
  auto out_at = [&](int r) {                                   // where matrix row r of the tile goes
    const int vr = mt * pl.RT + r / pl.G, s = seq_of(tab, vr);
    return (((int64_t)tab.row0[s] + vr - tab.cum[s]) * a.Hq + g * pl.G + r % pl.G) * HD + cb * CCOLS;
  };
  constexpr int CP = CCOLS / 2;
  int r = quad * 32 + threadIdx.x / CP;                        // the first row that this thread writes
  int64_t at = threadIdx.x < 32 * CP && r < rows ? out_at(r) : 0;
  wait_prerequisites();
  // this tile's parts lie nt apart, from p0 on
  const int64_t p0 = ((int64_t)g * pl.MP + mt / pl.nt) * pl.ns * pl.nt + mt % pl.nt;
  const float2* ml =
      reinterpret_cast<const float2*>((const float*)a.ws + (int64_t)pl.MP * a.Hkv * pl.ns * pl.nt * BQ * HD) +
      p0 * BQ + quad * 32 + lane;
  const float4* ps = reinterpret_cast<const float4*>(a.ws) + ((p0 * 4 + quad) * (HD / 4) + cb * (CCOLS / 4)) * 32 + lane;
  float m = -INFINITY, l = 0.f;
  float4 o[CCOLS / 4] = {};
  constexpr int U = 4;                                         // parts read together
  for (int p = w; p < pl.ns; p += U * W) {
    float2 x[U];
    float4 v[U][CCOLS / 4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      x[k] = make_float2(-INFINITY, 0.f);
      if (p + k * W < pl.ns) {
        x[k] = __ldcg(ml + (int64_t)(p + k * W) * pl.nt * BQ);
#pragma unroll
        for (int c = 0; c < CCOLS / 4; ++c) v[k][c] = __ldcg(ps + ((int64_t)(p + k * W) * pl.nt * HD + c) * 32);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (x[k].x == -INFINITY && x[k].y == 0.f) continue;
      const float M = fmaxf(m, x[k].x), wo = part_weight(m, M), wp = part_weight(x[k].x, M);
      m = M;
      l = wo * l + wp * x[k].y;
#pragma unroll
      for (int c = 0; c < CCOLS / 4; ++c) {
        o[c].x = wo * o[c].x + wp * v[k][c].x;
        o[c].y = wo * o[c].y + wp * v[k][c].y;
        o[c].z = wo * o[c].z + wp * v[k][c].z;
        o[c].w = wo * o[c].w + wp * v[k][c].w;
      }
    }
  }
  pml[w][lane] = make_float2(m, l);
#pragma unroll
  for (int c = 0; c < CCOLS / 4; ++c) po[w][c][lane] = o[c];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * CP; i += blockDim.x) {    // (row, 2 columns)
    const int lr = i / CP, cp = i % CP;
    if (i != threadIdx.x) {
      r = quad * 32 + lr;
      at = r < rows ? out_at(r) : 0;
    }
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
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(a.out + at + cp * 2) = t5::h2u(y0 * inv, y1 * inv);
  }
}

// One or two query tiles an item, and how many parts an item's key tiles are split into: the choice with
// the least estimated time (us, all constants measured): waves of CTAs x (key tiles per part + a CTA's fixed
// cost) and, when split, the join's launch and the sums that are written and read. A key tile takes 1.13 us
// with two query tiles and 0.66 with one, or as long as all CTAs' tiles need at 14 TB/s. Against the
// best of 80 forced choices, over 10 calls from 64 rows x 1024 to 1470 x 20000: within 8 %, mostly 3 %.
// (16 q heads, 128 rows over 2048: one part 19.2 us, seven 12.9; two tiles an item 28.1 and 14.1.) At most
// 64 parts, at most 8 CTAs an SM; and at least as many parts as keep each to LONGEST key tiles, whatever the
// estimate: the tensor cores add to one sum per output and drop what lies below its last bits (2^18, 2^20 keys of
// equal weight in one part: results 0.11, 0.61 percent low; in parts of at most LONGEST tiles 0.003 at both).
constexpr int LONGEST = 1024;
Plan make_plan(int V, int max_len, int P, int Hq, int Hkv, int hd, int num_sms) {
  Plan p;
  p.V = V;
  p.G = Hq / Hkv;
  p.RT = BQ / p.G;
  p.MT = (V + p.RT - 1) / p.RT;
  p.ncache = (int)(((int64_t)P + BKV - 1) / BKV);
  p.nt = p.ns = 1;
  p.MP = p.MT;
  double best = -1;
  for (int nt = 1; nt <= 2 && nt <= p.MT; ++nt) {
    const int64_t MP = (p.MT + nt - 1) / nt, items = MP * Hkv;
    const int64_t total = p.ncache + (std::min<int64_t>(V, (int64_t)max_len - 1 + nt * p.RT) + BKV - 1) / BKV;
    const int least = (int)std::min<int64_t>(64, (total + LONGEST - 1) / LONGEST);
    for (int ns = least; ns <= 64 && ns <= total && (ns == least || items * ns <= 8ll * num_sms); ++ns) {
      const int64_t ctas = items * ns;
      const double waves = (double)((ctas + num_sms - 1) / num_sms);
      const double l2 = (double)std::min<int64_t>(ctas, num_sms) * (4 * BKV) * hd / 14e6;
      double t = waves * (std::max(nt == 2 ? 1.13 : 0.66, l2) * (double)((total + ns - 1) / ns) + 4.5);
      if (ns > 1) t += 2.8 + 0.00006 * (double)(ctas * nt * hd);
      if (best < 0 || t < best) {
        best = t;
        p.nt = nt;
        p.MP = (int)MP;
        p.ns = ns;
      }
    }
  }
  return p;
}

// Packs sequences from `s` on into a table (empty ones left out) and returns the first one not taken.
int pack_group(SeqTab<SEQ_TAB_LARGE>& t, int s, int n_seq, const int* row0, const int* len, int* max_len) {
  t.n = 0;
  t.cum[0] = 0;
  *max_len = 0;
  for (; s < n_seq && t.n < SEQ_TAB_LARGE; ++s) {
    if (len[s] == 0) continue;
    if ((int64_t)t.cum[t.n] + len[s] > INT_MAX / 2) {
      if (t.n) break;
    }
    t.row0[t.n] = row0 ? row0[s] : 0;
    t.cum[t.n + 1] = t.cum[t.n] + len[s];
    *max_len = std::max(*max_len, len[s]);
    ++t.n;
  }
  return s;
}

template <int HD, bool E4M3, int N>
cudaError_t launch_group(const SharedAttnArgs& a, const SeqTab<N>& tab, const Plan& pl, const CUtensorMap& map,
                         cudaStream_t st) {
  using L = Lay<HD>;
  CK_RET(cudaFuncSetAttribute(shared_kernel<HD, E4M3, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  CK_RET(launch_pdl(shared_kernel<HD, E4M3, N>, dim3((unsigned)((int64_t)pl.MP * a.Hkv * pl.ns)), dim3(threads_of(E4M3)),
                    L::BYTES, st, tab, map, a, pl));
  if (pl.ns > 1) {
    const int warps = std::min(CWARPS, (pl.ns + 1) / 2);
    CK_RET(launch_pdl(combine_kernel<HD, N>, dim3((unsigned)((int64_t)pl.MT * a.Hkv * (HD / CCOLS * 4))),
                      dim3((unsigned)(32 * warps)), 0, st, tab, a, pl));
  }
  return cudaSuccess;
}

template <int N>
cudaError_t launch_tab(const SharedAttnArgs& a, const SeqTab<N>& tab, const Plan& pl, const CUtensorMap& map,
                       cudaStream_t st) {
  if (a.hd == 128)
    return a.e4m3 ? launch_group<128, true, N>(a, tab, pl, map, st) : launch_group<128, false, N>(a, tab, pl, map, st);
  return a.e4m3 ? launch_group<64, true, N>(a, tab, pl, map, st) : launch_group<64, false, N>(a, tab, pl, map, st);
}

}  // namespace sha

cudaError_t attention_shared_gave_up_word(uint64_t** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), sha::g_given_up);
}

int64_t attention_shared_ws_bytes(int n_seq, const int* len, int P, int Hq, int Hkv, int hd, int num_sms) {
  int64_t need = 0;
  SeqTab<SEQ_TAB_LARGE> t;
  for (int s = 0; s < n_seq;) {
    int max_len;
    s = sha::pack_group(t, s, n_seq, nullptr, len, &max_len);
    if (t.n == 0) continue;
    const sha::Plan p = sha::make_plan(t.cum[t.n], max_len, P, Hq, Hkv, hd, num_sms);
    if (p.ns > 1) need = std::max<int64_t>(need, (int64_t)p.MP * Hkv * p.ns * p.nt * sha::BQ * (hd + 2) * 4);
  }
  return need;
}

cudaError_t launch_attention_shared(const SharedAttnArgs& a, int n_seq, const int* row0, const int* len, int num_sms,
                                    cudaStream_t st) {
  CUtensorMap map = {};
  if (a.P > 0 && !a.e4m3) {
    // the P rows of each plane (rows past P read as zeros, never as what the capacity holds)
    const uint64_t dims[4] = {(uint64_t)a.hd, (uint64_t)a.Hkv, (uint64_t)a.P, 2};
    const uint64_t str[3] = {a.hd * 2ull, a.Hkv * a.hd * 2ull, (uint64_t)a.cap * a.Hkv * a.hd * 2};
    const uint32_t box[4] = {64, 1, sha::BKV, 1};
    if (!encode_tensor_map(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, a.kv, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  SeqTab<SEQ_TAB_LARGE> t;
  for (int s = 0; s < n_seq;) {
    int max_len;
    s = sha::pack_group(t, s, n_seq, row0, len, &max_len);
    if (t.n == 0) continue;
    const sha::Plan pl = sha::make_plan(t.cum[t.n], max_len, a.P, a.Hq, a.Hkv, a.hd, num_sms);
    if ((int64_t)pl.MP * a.Hkv * std::max(pl.ns, pl.nt * a.hd / 4) > INT_MAX) return cudaErrorInvalidValue;
    if (t.n <= SEQ_TAB_SMALL) {
      SeqTab<SEQ_TAB_SMALL> u;
      u.n = t.n;
      std::copy(t.cum, t.cum + t.n + 1, u.cum);
      std::copy(t.row0, t.row0 + t.n, u.row0);
      CK_RET(sha::launch_tab(a, u, pl, map, st));
    } else {
      CK_RET(sha::launch_tab(a, t, pl, map, st));
    }
  }
  return cudaSuccess;
}

}  // namespace s1
