// Attention of a batch of sequences over one shared prefix, on the 5th-generation tensor cores.
//
// Query row i of sequence s attends to the P rows of the snapshot and to rows 0 .. i of its own
// sequence: o = softmax(scale q.k) v. All sequences see the same prefix, so their query rows (and
// the G = Hq / Hkv q heads that share a kv head) are packed into tiles of 128 products' rows:
// RT = floor(128 / G) query rows x G heads per tile, whichever sequences the rows belong to. A
// tile reads each 128-key tile of the prefix once; s1_op_attention's kernel, one tile per
// (sequence, q head), would read it once per sequence and head.
//
// One pass over the keys with a running maximum and sum in fp32. Work items are (kv head, tile of
// query rows); when there are fewer items than SMs the key tiles of an item are split over `ns`
// CTAs whose (o, m, l) are joined in part order by combine_kernel (no atomics: the same bits every
// time). One CTA per SM, 14 warps:
//   warp 0      TMA producer: prefix tiles (f16 K/V tiles, or e4m3 tiles into a ring of raw stages)
//   warp 1      TMEM allocation, MMA issue: S = Q K^T into one of two TMEM buffers, O += P V with P
//               read from TMEM (f16, written by the softmax warps; no shared-memory round trip)
//   warps 2-9   softmax, two threads per row (64 keys each): mask, running max with a lazy rescale
//               (O and l move only when the row's maximum grows by more than 2^8), P back to TMEM;
//               warps whose 32 rows are all past the tile's last row only keep the barriers going
//   warps 10-13 loaders: the batch's own keys (gathered row by row through the sequence table), and
//               e4m3 prefix tiles: codes from the raw stage to f16 in the MMA's swizzled layout
// Own keys are packed the same way as queries: row r's visible own keys are the packed rows
// start(r) .. r, so one masked tile serves many short sequences. A masked weight is an exact zero,
// but 0 x NaN is not: the loaders replace non-finite own V elements by 0 and flag the tile, and
// the epilogue of a flagged tile adds them to exactly the rows that see them.
// An e4m3 code times its scale is exact in f16 for scales 2^-6 .. 2^7 (and rounded as the read-back
// rounds it otherwise), so the products run on f16 operands as with an f16 snapshot.
// Every mbarrier wait is bounded; on expiry an error word is set and every role leaves.
#include <algorithm>
#include <climits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace sha {
using namespace t5;

constexpr int BQ = 128, BKV = 128;
constexpr int NTHREADS = 14 * 32;
constexpr int ST = 2;                        // f16 K and V stages
constexpr int RS = 3;                        // raw e4m3 stages (K and V tiles in turn)
constexpr int TMEM_COLS = 512;               // S 2 x 128 | O hd at 256 | P 2 x 64 at 384
constexpr int T_O = 256, T_P = 384;
constexpr int ERR_TIMEOUT = 0x401;

__device__ int g_err;                        // bounded waits record here (one word per device)

struct Plan {
  int V;          // packed query rows
  int G, RT, MT;  // q heads per kv head, query rows per tile, tiles
  int ns;         // key parts per item
  int ncache;     // prefix tiles
};

template <int HD, bool E4M3>
struct Lay {
  static constexpr int TILE = BKV * HD * 2;
  static constexpr int RAW = BKV * HD;
  static constexpr int Q = 0;                             // HD/64 boxes of [128 rows][128 B]
  static constexpr int K = Q + BQ * HD * 2;
  static constexpr int V = K + ST * TILE;
  static constexpr int R = V + ST * TILE;
  static constexpr int XCH = R + (E4M3 ? RS * RAW : 0);   // row maxima / sums of the halves [3][2][BQ]
  static constexpr int BAR = XCH + 3 * 2 * BQ * 4;
  static constexpr int USED = BAR + 512 + 1024;           // barriers, alignment slack
  // above half an SM: each CTA allocates all of TMEM, so two never share one
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
};

// The sequence that packed row vr (< cum[n]) belongs to.
template <int N>
__device__ __forceinline__ int seq_of(const SeqTab<N>& t, int vr) {
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

// Sixteen e4m3 codes times scale to f16 (round to nearest even, held at +-65504). fast: the scale
// is an f16 value of at most 2^7, so the f16 product is the rounded value and cannot overflow.
__device__ __forceinline__ void codes_to_half(const uint4 c, float scale, bool fast, uint32_t* h) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const __half2 s2 = __float2half2_rn(scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 x = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    __half2 y;
    if (fast) {
      y = __hmul2(x, s2);
    } else {
      const float2 f = __half22float2(x);
      const float a = f.x * scale, b = f.y * scale;
      y = __floats2half2_rn(fabsf(a) > 65504.f ? copysignf(65504.f, a) : a,
                            fabsf(b) > 65504.f ? copysignf(65504.f, b) : b);
    }
    h[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <int HD, bool E4M3, int N>
__global__ void __launch_bounds__(NTHREADS, 1)
    shared_kernel(const __grid_constant__ SeqTab<N> tab, const __grid_constant__ CUtensorMap mapKV,
                  const __grid_constant__ SharedAttnArgs a, const Plan pl) {
  using L = Lay<HD, E4M3>;
  constexpr int NB = HD / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(sm + L::BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;                 // [ST]
  uint64_t* v_full = k_full + ST;              // [ST]
  uint64_t* k_empty = v_full + ST;             // [ST]
  uint64_t* v_empty = k_empty + ST;            // [ST]
  uint64_t* s_full = v_empty + ST;             // [2]
  uint64_t* s_empty = s_full + 2;              // [2]
  uint64_t* p_full = s_empty + 2;              // [2]
  uint64_t* o_done = p_full + 2;               // [2]
  uint64_t* mma_idle = o_done + 2;
  uint64_t* xbar = mma_idle + 1;               // [4 quadrants][3]: the two warps of a row quadrant meet
  uint64_t* raw_full = xbar + 12;              // [RS]
  uint64_t* raw_empty = raw_full + RS;         // [RS]
  uint32_t* tmem_slot = (uint32_t*)(raw_empty + RS);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* v_flag = (volatile int*)(tmem_slot + 2);   // some own V element of this CTA is not finite
  static_assert((1 + 4 * ST + 9 + 12 + 2 * RS) * 8 + 16 <= 512, "barriers fit");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % pl.ns), item = (int)(blockIdx.x / pl.ns);
  const int mt = item % pl.MT, g = item / pl.MT;
  const int v0 = mt * pl.RT;                   // first packed row of the tile, and one past its last
  const int v1 = min(pl.V, v0 + pl.RT);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], E4M3 ? 4 : 5);
      mbar_init(&v_full[s], E4M3 ? 4 : 5);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], 8);
      mbar_init(&p_full[b], 8);
      mbar_init(&o_done[b], 1);
    }
    mbar_init(mma_idle, 1);
    for (int x = 0; x < 12; ++x) mbar_init(&xbar[x], 2);
    for (int r = 0; r < RS; ++r) { mbar_init(&raw_full[r], 1); mbar_init(&raw_empty[r], 4); }
    *abort_flag = 0;
    *v_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<TMEM_COLS>(tmem_slot);
  allow_dependents();
  wait_prerequisites();
  // key tiles of this part: prefix tiles 0 .. ncache-1, then own tiles from packed row kb on
  const int kb = a.kn ? tab.cum[seq_of(tab, v0)] : 0;
  const int nown = a.kn ? (v1 - kb + BKV - 1) / BKV : 0;
  const int total = pl.ncache + nown;
  const int per = (total + pl.ns - 1) / pl.ns;
  const int jb = min(total, part * per), je = min(total, jb + per);
  const int n = je - jb;
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---- TMA producer
    if (lane == 0) {
      int i = 0;
      if constexpr (E4M3) {
        int it = 0;                            // raw items issued: K and V tiles in turn
        bool ok = true;
        for (; i < n && jb + i < pl.ncache && ok; ++i)
          for (int pln = 0; pln < 2 && ok; ++pln, ++it) {
            const int r = it % RS;
            ok = mbar_wait(&raw_empty[r], ((it / RS) & 1) ^ 1, abort_flag, &g_err, ERR_TIMEOUT);
            if (!ok) break;
            mbar_expect_tx(&raw_full[r], L::RAW);
            tma4(sm + L::R + r * L::RAW, &mapKV, &raw_full[r], 0, g, (jb + i) * BKV, pln);
          }
        if (*abort_flag)                       // copies in flight land before the CTA leaves
          for (int x = it > RS ? it - RS : 0; x < it; ++x) mbar_drain(&raw_full[x % RS], (x / RS) & 1);
      } else {
        bool ok = true;
        int ki = 0, vi = 0;                    // fills begun
        for (; i < n && ok; ++i) {
          const int s = i % ST, j = jb + i;
          const uint32_t ph = ((i / ST) & 1) ^ 1;
          ok = mbar_wait(&k_empty[s], ph, abort_flag, &g_err, ERR_TIMEOUT);
          if (!ok) break;
          if (j < pl.ncache) {
            mbar_expect_tx(&k_full[s], L::TILE);
            for (int b = 0; b < NB; ++b)
              tma4(sm + L::K + s * L::TILE + b * BKV * 128, &mapKV, &k_full[s], 64 * b, g, j * BKV, 0);
          } else {
            mbar_arrive(&k_full[s]);
          }
          ki = i + 1;
          ok = mbar_wait(&v_empty[s], ph, abort_flag, &g_err, ERR_TIMEOUT);
          if (!ok) break;
          if (j < pl.ncache) {
            mbar_expect_tx(&v_full[s], L::TILE);
            for (int b = 0; b < NB; ++b)
              tma4(sm + L::V + s * L::TILE + b * BKV * 128, &mapKV, &v_full[s], 64 * b, g, j * BKV, 1);
          } else {
            mbar_arrive(&v_full[s]);
          }
          vi = i + 1;
        }
        if (*abort_flag) {
          for (int x = ki > ST ? ki - ST : 0; x < ki; ++x) mbar_drain(&k_full[x % ST], (x / ST) & 1);
          for (int x = vi > ST ? vi - ST : 0; x < vi; ++x) mbar_drain(&v_full[x % ST], (x / ST) & 1);
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer
    if (lane == 0 && n > 0) {
      constexpr uint32_t ID_S = idesc_f16(BKV, 0, 0, 0), ID_O = idesc_f16(HD, 0, 0, 1);
      bool ok = mbar_wait(q_full, 0, abort_flag, &g_err, ERR_TIMEOUT);
      auto issue_s = [&](int i) -> bool {      // S_i = Q K_i^T into buffer i & 1
        const int s = i % ST, b = i & 1;
        if (!mbar_wait(&k_full[s], (i / ST) & 1, abort_flag, &g_err, ERR_TIMEOUT)) return false;
        if (!mbar_wait(&s_empty[b], ((i >> 1) & 1) ^ 1, abort_flag, &g_err, ERR_TIMEOUT)) return false;
        fence_after();
        const uint32_t qa = smem_u32(sm + L::Q), ka = smem_u32(sm + L::K + s * L::TILE);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (uint32_t)((kk >> 2) * (128 * 128) + (kk & 3) * 32);
          mma_ss(tmem + b * 128, desc_sw128(qa + off, 16), desc_sw128(ka + off, 16), ID_S, kk > 0 ? 1u : 0u);
        }
        commit(&s_full[b]);
        commit(&k_empty[s]);
        return true;
      };
      auto issue_pv = [&](int i) -> bool {     // O += P_i V_i
        const int s = i % ST, b = i & 1;
        if (!mbar_wait(&p_full[b], (i >> 1) & 1, abort_flag, &g_err, ERR_TIMEOUT)) return false;
        if (!mbar_wait(&v_full[s], (i / ST) & 1, abort_flag, &g_err, ERR_TIMEOUT)) return false;
        fence_after();
        const uint32_t va = smem_u32(sm + L::V + s * L::TILE);
#pragma unroll
        for (int kk = 0; kk < BKV / 16; ++kk)
          mma_ts(tmem + T_O, tmem + T_P + b * 64 + kk * 8, desc_sw128(va + kk * 16 * 128, BKV * 128), ID_O,
                 (i > 0 || kk > 0) ? 1u : 0u);
        commit(&o_done[b]);
        commit(&v_empty[s]);
        return true;
      };
      if (ok) ok = issue_s(0);
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n) ok = issue_s(i + 1);
        if (ok) ok = issue_pv(i);
      }
      commit(mma_idle);
      mbar_drain(mma_idle, 0);                 // every MMA issued above has completed
    }
  } else if (warp >= 10) {
    // ---- loaders: rows 32 lw .. +31 of every tile
    const int lw = warp - 10;
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_err, ERR_TIMEOUT) ? 1 : 0) != 0;
    };
    auto publish = [&](uint64_t* bar) {        // this warp's writes to shared memory are the MMA's to read
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
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
#pragma unroll
      for (int p0 = 0; p0 < PASSES; p0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int p = 0; p < 8 && p0 + p < PASSES; ++p) {
          const int64_t o = __shfl_sync(0xffffffffu, off, (p0 + p) * RPI + lane / CH);
          x[p] = o >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + o) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < 8 && p0 + p < PASSES; ++p) {
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
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % ST, j = jb + i;
      const uint32_t ph = ((i / ST) & 1) ^ 1;
      const bool cache = j < pl.ncache;
#pragma unroll
      for (int pln = 0; pln < 2; ++pln) {
        uint64_t* empty = pln ? &v_empty[s] : &k_empty[s];
        uint64_t* full = pln ? &v_full[s] : &k_full[s];
        uint8_t* dst = sm + (pln ? L::V : L::K) + s * L::TILE;
        if (!cache) {
          ok = wwait(empty, ph);
          if (!ok) break;
          load_own(j - pl.ncache, pln ? a.vn : a.kn, dst, pln == 1);
        } else if constexpr (E4M3) {
          const int it = 2 * i + pln, r = it % RS;
          const int key = j * BKV + lw * 32 + lane;
          const float sc = key < a.P ? a.scales[((int64_t)pln * a.Hkv + g) * a.cap + key] : 1.f;
          const bool fast = __all_sync(0xffffffffu, sc <= 128.f && __half2float(__float2half_rn(sc)) == sc);
          ok = wwait(&raw_full[r], (it / RS) & 1) && wwait(empty, ph);
          if (!ok) break;
          // LPR lanes of 16 codes per row; the lanes of a row's second 64 columns (or of odd rows)
          // write their two 16-byte chunks in the other order, so that no store conflicts
          constexpr int LPR = HD / 16, RP = 32 / LPR;
          const int ci = lane % LPR;
          const uint8_t* raw = sm + L::R + r * L::RAW + (lw * 32) * HD + lane * 16;
#pragma unroll 4
          for (int p = 0; p < 32 / RP; ++p) {
            const int lr = p * RP + lane / LPR, row = lw * 32 + lr;
            const uint4 c = *reinterpret_cast<const uint4*>(raw + p * RP * HD);
            uint32_t h[8];
            codes_to_half(c, __shfl_sync(0xffffffffu, sc, lr), fast, h);
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            const bool swap = HD == 128 && ci >= 4;
            uint8_t* d = dst + (ci >> 2) * (BKV * 128) + row * 128;
            const int c0 = (2 * ci) & 7;
            *reinterpret_cast<uint4*>(d + (((c0 + (swap ? 1 : 0)) ^ (row & 7)) << 4)) = swap ? hi : lo;
            *reinterpret_cast<uint4*>(d + (((c0 + (swap ? 0 : 1)) ^ (row & 7)) << 4)) = swap ? lo : hi;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[r]);
        } else {
          ok = wwait(empty, ph);               // the producer's tile: only the arrival
          if (!ok) break;
        }
        publish(full);
      }
    }
  } else {
    // ---- softmax: row r = TMEM lane r; warps 2-5 keys 0..63 of a tile, warps 6-9 keys 64..127
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_err, ERR_TIMEOUT) ? 1 : 0) != 0;
    };
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int r = quad * 32 + lane;
    const int vq = v0 + r / pl.G;              // packed query row of this row
    const bool live = r < pl.RT * pl.G && vq < v1;
    const int h = g * pl.G + r % pl.G;
    int vs = 0;
    int64_t row = -1;                          // row of q and out
    if (live) {
      const int s = seq_of(tab, vq);
      vs = tab.cum[s];
      row = (int64_t)tab.row0[s] + (vq - vs);
    }
    const bool idle = !__any_sync(0xffffffffu, live);   // (the same for both halves of a quadrant)
    {   // Q rows of the quadrant: half 0 the row's first chunks, half 1 the rest; absent rows are zeros
      constexpr int CHH = HD / 16, RPI = 32 / CHH;      // 16-byte chunks of a half row
      const int64_t off = live ? row * a.q_stride + (int64_t)h * HD : -1;
      const int c = half * CHH + lane % CHH;
      uint4 x[32 / RPI];
#pragma unroll
      for (int p = 0; p < 32 / RPI; ++p) {
        const int64_t o = __shfl_sync(0xffffffffu, off, p * RPI + lane / CHH);
        x[p] = o >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + o) + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int p = 0; p < 32 / RPI; ++p) {
        const int rr = quad * 32 + p * RPI + lane / CHH;
        *reinterpret_cast<uint4*>(sm + L::Q + (c >> 3) * (BQ * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = x[p];
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_off + T_O + (uint32_t)(half * (HD / 2));
    float* xch = reinterpret_cast<float*>(sm + L::XCH);
    auto pair_meet = [&](int slot, uint32_t parity) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&xbar[quad * 3 + slot]);
      return wwait(&xbar[quad * 3 + slot], parity);
    };
    constexpr int HB = BKV / 2, HO = HD / 2;
    const float sl2 = a.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.f;              // maximum (log2 domain), this half's share of the sum
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int j = jb + i, b = i & 1;
      const uint32_t ph = (i >> 1) & 1;
      if (!wwait(&s_full[b], ph)) { ok = false; break; }
      if (idle) {
        if (lane == 0) mbar_arrive(&s_empty[b]);
        if (i >= 2 && !wwait(&o_done[b], ph ^ 1)) { ok = false; break; }
        if (lane == 0) mbar_arrive(&p_full[b]);
        continue;
      }
      fence_after();
      uint32_t u[HB];
      tld32(tmem + lane_off + b * 128 + half * HB, u);
      tld32(tmem + lane_off + b * 128 + half * HB + 32, u + 32);
      ld_wait();
      pin32(u);
      pin32(u + 32);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[b]);
      // visible keys of this half tile: lo .. hi
      int lo = 0, hi;
      if (j < pl.ncache) {
        hi = a.P - 1 - j * BKV - half * HB;
      } else {
        const int base = kb + (j - pl.ncache) * BKV + half * HB;
        lo = vs - base;
        hi = live ? vq - base : -1;
      }
      float mx = -INFINITY;
      if (__all_sync(0xffffffffu, lo <= 0 && hi >= HB - 1)) {
#pragma unroll
        for (int c = 0; c < HB; ++c) mx = fmaxf(mx, __uint_as_float(u[c]));
      } else {
#pragma unroll
        for (int c = 0; c < HB; ++c) {
          if (c < lo || c > hi) u[c] = 0xff800000u;
          mx = fmaxf(mx, __uint_as_float(u[c]));
        }
      }
      xch[(b * 2 + half) * BQ + r] = mx;
      if (!pair_meet(b, ph)) { ok = false; break; }
      mx = fmaxf(mx, xch[(b * 2 + (half ^ 1)) * BQ + r]) * sl2;
      float alpha = 1.f;
      if (mx > m + 8.f) {
        alpha = m == -INFINITY ? 1.f : ex2(m - mx);
        m = mx;
      }
      const float base = m == -INFINITY ? 0.f : m;
      if (i >= 2 && !wwait(&o_done[b], ph ^ 1)) { ok = false; break; }         // P_{i-2} has been read
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!wwait(&o_done[b ^ 1], ((i - 1) >> 1) & 1)) { ok = false; break; }   // O holds P_{i-1} V_{i-1}
        fence_after();
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < HO; c += 32) {
          tld32(tO + c, w);
          ld_wait();
          pin32(w);
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
          tst32(tO + c, w);
        }
        l *= alpha;
      }
      fence_after();
      float rs = 0.f;
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < HB; c += 2) {
        const float p0 = ex2(fmaf(__uint_as_float(u[c]), sl2, -base));
        const float p1 = ex2(fmaf(__uint_as_float(u[c + 1]), sl2, -base));
        rs += p0 + p1;
        pk[c / 2] = h2u(p0, p1);
      }
      l += rs;
      tst32(tmem + lane_off + T_P + b * 64 + half * 32, pk);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[b]);
    }
    // ---- epilogue: each thread its half of the row's output columns
    if (ok && n > 0) ok = wwait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (!idle) {
      xch[(2 * 2 + half) * BQ + r] = l;
      if (pair_meet(2, 0)) l += xch[(2 * 2 + (half ^ 1)) * BQ + r];
      else ok = false;
      float o[HO];
      if (ok && n > 0) {
        fence_after();
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < HO; c += 32) {
          tld32(tO + c, w);
          ld_wait();
          pin32(w);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[c + e] = __uint_as_float(w[e]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < HO; ++c) o[c] = 0.f;
      }
      if (ok && live && *v_flag) {             // non-finite own V elements: into the rows that see them
        const int k0 = max(vs, kb + (max(jb, pl.ncache) - pl.ncache) * BKV);
        const int k1 = min(vq, kb + (je - pl.ncache) * BKV - 1);
        for (int kv = k0; kv <= k1; ++kv) {
          const f16* vp = a.vn + (row - (vq - kv)) * a.kv_stride + (int64_t)g * HD + half * HO;
#pragma unroll
          for (int c = 0; c < HO; ++c) {
            const float x = h2f(vp[c]);
            if (!isfinite(x)) o[c] += x;
          }
        }
      }
      if (ok && live) {
        if (pl.ns == 1) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          f16* op = a.out + (row * a.Hq + h) * HD + half * HO;
#pragma unroll
          for (int c = 0; c < HO; c += 8)
            *reinterpret_cast<uint4*>(op + c) =
                make_uint4(h2u(o[c] * inv, o[c + 1] * inv), h2u(o[c + 2] * inv, o[c + 3] * inv),
                           h2u(o[c + 4] * inv, o[c + 5] * inv), h2u(o[c + 6] * inv, o[c + 7] * inv));
        } else {                               // [items * ns][BQ][HD] sums, then [..][BQ] (m, l)
          const int64_t pi = (int64_t)blockIdx.x * BQ + r;
          float* wo = (float*)a.ws + pi * HD + half * HO;
#pragma unroll
          for (int c = 0; c < HO; c += 4)
            *reinterpret_cast<float4*>(wo + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          if (half == 0)
            reinterpret_cast<float2*>((float*)a.ws + (int64_t)gridDim.x * BQ * HD)[pi] = make_float2(m, l);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<TMEM_COLS>(tmem);
  }
}

// Joins the parts of a row in part order: M = max m, o = sum 2^(m - M) o / sum 2^(m - M) l. One
// warp per (packed row, q head). A part without a visible key (m = -inf, l = 0) holds no sums.
template <int HD, int N>
__global__ void __launch_bounds__(256)
    combine_kernel(const __grid_constant__ SeqTab<N> tab, const __grid_constant__ SharedAttnArgs a, const Plan pl) {
  constexpr int E = HD / 32;
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int vr = (int)(w / a.Hq), h = (int)(w % a.Hq);
  if (vr >= pl.V) return;
  const int g = h / pl.G, mt = vr / pl.RT;
  const int r = (vr - mt * pl.RT) * pl.G + h % pl.G;
  const int64_t p0 = ((int64_t)g * pl.MT + mt) * pl.ns;        // the item's first part
  const float2* ml = reinterpret_cast<const float2*>((const float*)a.ws + (int64_t)pl.MT * a.Hkv * pl.ns * BQ * HD);
  const float* po = (const float*)a.ws + (p0 * BQ + r) * HD + lane * E;
  float2 x[2];                                                 // ns <= 64: parts lane and lane + 32
  float M = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int p = lane + 32 * k;
    x[k] = p < pl.ns ? ml[(p0 + p) * BQ + r] : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, x[k].x);
  }
  M = warp_max(M);
  float sum = 0.f, wt[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    wt[k] = x[k].x == -INFINITY && x[k].y == 0.f ? 0.f : t5::ex2(x[k].x - M);
    sum += wt[k] == 0.f && x[k].y == 0.f ? 0.f : wt[k] * x[k].y;
  }
  sum = warp_sum(sum);
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const unsigned used0 = __ballot_sync(0xffffffffu, !(x[0].x == -INFINITY && x[0].y == 0.f));
  const unsigned used1 = __ballot_sync(0xffffffffu, !(x[1].x == -INFINITY && x[1].y == 0.f));
#pragma unroll 4
  for (int p = 0; p < pl.ns; ++p) {
    const float f = __shfl_sync(0xffffffffu, p < 32 ? wt[0] : wt[1], p & 31);
    if (!(((p < 32 ? used0 : used1) >> (p & 31)) & 1)) continue;
    const float* op = po + (int64_t)p * BQ * HD;
    float v[E];
    if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(op);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(op);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += f * v[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int s = seq_of(tab, vr);
  f16* out = a.out + (((int64_t)tab.row0[s] + vr - tab.cum[s]) * a.Hq + h) * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(out + e) = t5::h2u(o[e] * inv, o[e + 1] * inv);
}

// How many parts an item's key tiles are split into: the count with the least time in units of one
// key tile, (waves of CTAs) x (tiles per part + a CTA's fixed cost of about 4 tiles), plus, when
// split, the join's launch and its reads of the parts. At most 64 parts, at most 8 CTAs an SM.
Plan make_plan(int V, int max_len, int P, int Hq, int Hkv, int num_sms) {
  Plan p;
  p.V = V;
  p.G = Hq / Hkv;
  p.RT = BQ / p.G;
  p.MT = (V + p.RT - 1) / p.RT;
  p.ncache = (int)(((int64_t)P + BKV - 1) / BKV);
  const int64_t items = (int64_t)p.MT * Hkv;
  const int64_t total = p.ncache + (std::min<int64_t>(V, (int64_t)max_len - 1 + p.RT) + BKV - 1) / BKV;
  p.ns = 1;
  double best = 0;
  for (int ns = 1; ns <= 64 && ns <= total && (ns == 1 || items * ns <= 8ll * num_sms); ++ns) {
    const double waves = (double)((items * ns + num_sms - 1) / num_sms);
    double t = waves * ((double)((total + ns - 1) / ns) + 4.0);
    if (ns > 1) t += 5.0 + 0.02 * (double)(items * ns);
    if (ns == 1 || t < best) {
      best = t;
      p.ns = ns;
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
  using L = Lay<HD, E4M3>;
  CK_RET(cudaFuncSetAttribute(shared_kernel<HD, E4M3, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  CK_RET(launch_pdl(shared_kernel<HD, E4M3, N>, dim3((unsigned)((int64_t)pl.MT * a.Hkv * pl.ns)), dim3(NTHREADS),
                    L::BYTES, st, tab, map, a, pl));
  if (pl.ns > 1) {
    const int64_t warps = (int64_t)pl.V * a.Hq;
    CK_RET(launch_pdl(combine_kernel<HD, N>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, tab, a, pl));
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

cudaError_t op_error_word(int** out) { return cudaGetSymbolAddress(reinterpret_cast<void**>(out), sha::g_err); }

int64_t attention_shared_ws_bytes(int n_seq, const int* len, int P, int Hq, int Hkv, int hd, int num_sms) {
  int64_t need = 0;
  SeqTab<SEQ_TAB_LARGE> t;
  for (int s = 0; s < n_seq;) {
    int max_len;
    s = sha::pack_group(t, s, n_seq, nullptr, len, &max_len);
    if (t.n == 0) continue;
    const sha::Plan p = sha::make_plan(t.cum[t.n], max_len, P, Hq, Hkv, num_sms);
    if (p.ns > 1) need = std::max<int64_t>(need, (int64_t)p.MT * Hkv * p.ns * sha::BQ * (hd + 2) * 4);
  }
  return need;
}

cudaError_t launch_attention_shared(const SharedAttnArgs& a, int n_seq, const int* row0, const int* len, int num_sms,
                                    cudaStream_t st) {
  CUtensorMap map = {};
  if (a.P > 0) {
    // the P rows of each plane (rows past P read as zeros, never as what the capacity holds)
    const uint64_t es = a.e4m3 ? 1 : 2;
    const uint64_t dims[4] = {(uint64_t)a.hd, (uint64_t)a.Hkv, (uint64_t)a.P, 2};
    const uint64_t str[3] = {a.hd * es, (uint64_t)a.Hkv * a.hd * es, (uint64_t)a.cap * a.Hkv * a.hd * es};
    const uint32_t box[4] = {a.e4m3 ? (uint32_t)a.hd : 64u, 1, sha::BKV, 1};
    if (!encode_tensor_map(&map, a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, a.kv,
                           dims, str, box, a.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  SeqTab<SEQ_TAB_LARGE> t;
  for (int s = 0; s < n_seq;) {
    int max_len;
    s = sha::pack_group(t, s, n_seq, row0, len, &max_len);
    if (t.n == 0) continue;
    const sha::Plan pl = sha::make_plan(t.cum[t.n], max_len, a.P, a.Hq, a.Hkv, num_sms);
    if ((int64_t)pl.MT * a.Hkv * pl.ns > INT_MAX) return cudaErrorInvalidValue;
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
