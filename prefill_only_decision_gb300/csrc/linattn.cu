// Linear attention with a decay per head: S_t = lam_h S_{t-1} + v_t k_t^T, o_t = scale S_t q_t,
// lam_h = exp(log_decay[h]). Prompts (launch_linattn) and single tokens (launch_linattn_step).
//
// Prompts run in chunks of 128 rows on the 5th-generation tensor cores. Within a chunk of n rows,
// with S the state before it:
//   O  = diag(scale lam^(i+1)) Q S^T + (scale lam^(i-j) q_i.k_j for j <= i, else 0) V
//   S' = lam^n S + sum_j (lam^(n-1-j) v_j) k_j^T
// One CTA takes a segment of consecutive chunks of one (sequence, head) in order, the state in TMEM
// (fp32, lane = value row). A call with too few (sequence, head) pairs for the GPU cuts sequences
// into segments: a first launch forms every segment's own contribution to the state (the second
// line alone, from zero), a second joins them into the segments' start states, a third is the
// pass over the chunks. What bounds it: q, k, v read and o written once, 4 x 32 KB per chunk and
// head at 128 x 128, about 2.9 us of an SM's share of the HBM rate; the products of a chunk take
// about 1.3 us of tensor time. Measured: 4.0 us a chunk with all SMs busy (the chain of the state from
// chunk to chunk through two products and two passes of the value-row warps) and 6 us before the first
// and behind the last; 1024 rows x 16 heads f16 21.7 us, 16476 x 32 bf16 189 us, f16
// 217 (its reads and writes alone: 81); 64 x 64, 16476 x 32 bf16 151, f16 180 (40).
// Operand precision: products take 16-bit operands and sum in fp32. Q, K and V enter as given: of a row's
// decay lam^(i+1) = 2^e r, Q takes 2^e (exact), the outputs r in fp32, the weights 1 / r with their own
// decay (a rounded decayed Q put the outputs' error at 1.57 x one rounding to the rows' type, instead of
// 1.41). The weights of V in a chunk and the state's operand copy are rounded once to the rows' type (the
// state itself never is). The decayed values v_j lam^(n-1-j) of the state update are split into such
// numbers, because the state is kept and returned in fp32: two for f16 (they leave 5e-8), three for bf16
// (two leave 2.5e-6, three put the state's error at 3e-7, most of it fp32's, and took 16476 rows x 32
// heads from 182 to 202 us, 188 since they wait for no more than they must). Their products run small
// parts first: the sums lose less.
// f16 rows: weights, scaled Q and the state's copy are scaled by powers of two so that they use f16's range whatever
// the magnitudes: the state's copy by 2^a (from a running bound on the state before the chunk, to which each row adds
// lam^(n-1-j) max|v_j| max|k_j|), a row's weights by 2^c, its Q by 2^(c - a) and its outputs by 2^-c, with c from the
// row's own largest weight and largest |q|: a row's scales depend on nothing that it does not see, and a large
// element costs only rows that have it in their sums anyway. (c for 32 rows at once from dk max|q| max|k| of the
// whole chunk, and a bound that grew by n max|v| max|k| a chunk, needed a pass over the weights less, 16384 rows x 32
// heads 212 us instead of 218, 8000 x 16 of 64 52 instead of 58; but a key of 4000 in a later row cost ordinary
// rows before it percents, and so did elements of 9000 rows after them where the decay had long forgotten them.)
// What lies 2^28 below a row's largest weight, or below the bound, loses bits: an output whose values are all zeros
// next to such a weight keeps less of what the state gives it (bf16 has no such limit).
// The decayed values, with the state they are added to, are scaled by 2^b (b per chunk, from its largest decayed
// value), so that the low parts stay above f16's smallest number: a decayed value keeps 2^-24 of itself down to 2^-13
// of the chunk's largest, and is off by at most 2^-37 of that below.
// Where: f16's scaled Q is in TMEM beside the weights; bf16's is in its shared-memory tile, and the third
// parts take its TMEM columns (so they wait for the weights, and the next Q K^T waits for them).
// One CTA per SM, 23 warps: 0 TMA producer (two stages of Q, K, V); 1 and 18 MMA issue (1: Q K^T and
// the outputs, 18: the state); 2-9 rows of the chunk (TMEM lane = row, two threads a row: weights,
// scaled Q); 10-17 value rows (TMEM lane = value row, two threads a row: the split decayed values,
// the state's copy and decay); 19-22 outputs (a thread a row). Their passes are loops over 32
// columns, not unrolled code: a chunk's worth of straight-line code per role does not stay in the
// instruction cache, and took longer.
// 0 x NaN: rows past the sequence are zeroed in shared memory; non-finite V elements are replaced
// by 0 and their terms are added, in the plain order of the formula, to exactly the rows and state
// rows that they belong to.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace s1 {
namespace lin {
using namespace t5;

__device__ __forceinline__ float ld_f(const f16* p) { return __half2float(*p); }
__device__ __forceinline__ float ld_f(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_f(f16* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void st_f(bf16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ uint32_t pack(f16, float lo, float hi) { return h2u(lo, hi); }
__device__ __forceinline__ uint32_t pack(bf16, float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack(f16, uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ float2 unpack(bf16, uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// an element's exponent field is all ones
__device__ __forceinline__ bool nonfinite(f16, uint32_t u16) { return (u16 & 0x7c00u) == 0x7c00u; }
__device__ __forceinline__ bool nonfinite(bf16, uint32_t u16) { return (u16 & 0x7f80u) == 0x7f80u; }

// A head's log decay, at most 0; NaN stays NaN (fminf would make it no decay).
__device__ __forceinline__ float capped(float log_decay) { return log_decay > 0.f ? 0.f : log_decay; }
// log2 of a head's decay: at most 0, and never -inf (2^-1e4 is 0 as well, and 0 * -1e4 is 0)
__device__ __forceinline__ float log2_decay(float log_decay) {
  const float l2 = capped(log_decay) * 1.4426950408889634f;
  return l2 < -1e4f ? -1e4f : l2;
}
// exp of a head's log decay: at most 1, exactly 0 for -inf
__device__ __forceinline__ float decay(float log_decay) { return expf(capped(log_decay)); }

constexpr int C = 128;                       // rows of a chunk
constexpr int NTHREADS = 23 * 32;

__device__ uint64_t g_given_up;              // when a bounded wait last gave up, per device; never cleared

constexpr int MAX_SEQ = 256;                 // sequences per launch

// The sequences of a launch: rows row0[s] .. + len[s] - 1, cut into segments of seg_rows rows.
// Sequence s has fullcum[s+1] - fullcum[s] segments of that length, then possibly a shorter last one
// (an empty sequence has one of no rows): blocks take all full segments first, then the short ones,
// tailcum[s] of them before sequence s's. ws_seg[s]: the sequence's first start state in the
// workspace, or -1 when it has a single segment.
struct Tab {
  int n, seq0, seg_rows;
  int split;                                   // some sequence has several segments
  int fullcum[MAX_SEQ + 1], tailcum[MAX_SEQ + 1];
  int row0[MAX_SEQ], len[MAX_SEQ], ws_seg[MAX_SEQ];
};
// The entry that index i falls into: cum[s] <= i < cum[s + 1].
__device__ __forceinline__ int find(const int* cum, int n, int i) {
  int lo = 0, hi = n;                          // cum[lo] <= i < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// TMEM columns: weights of V, per half of 64 columns: fp32, then 16-bit in its first 32 columns and
// the half's scaled Q (f16) or third parts of the decayed values (bf16) in its last 32 | outputs | state |
// low and high parts of the decayed values
constexpr int TMEM_COLS = 512;
constexpr int T_P = 0, T_O = 128, T_S = 256, T_VL = 384, T_VH = 448;

template <int DK, int DV>
struct Lay {
  static constexpr int QB = C * DK * 2, VB = C * DV * 2;   // bytes of a Q or K tile, of a V tile
  static constexpr int STAGE = 2 * QB + VB;                // Q, K, V
  static constexpr int S16 = 2 * STAGE;                    // the state's operand copy [DV][DK]
  static constexpr int WV = S16 + DV * DK * 2 + 16;        // lam^(127-t), t = -1 .. 127; the same for the last
                                                           // chunk's length, t = 0 .. 127
  static constexpr int BAR = WV + 2 * C * 4;
  static constexpr int NBAR = 33;
  static constexpr int USED = BAR + NBAR * 8 + 13 * 4 + 12 * C;
  static_assert(USED <= 227 * 1024, "shared memory of one CTA");
  // above half an SM: each CTA allocates all of TMEM, so two never share one
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
};

// Smallest e with |x| < 2^e (finite x != 0).
__device__ __forceinline__ int exp_above(float x) { return (int)((__float_as_uint(x) >> 23) & 255) - 126; }
__device__ __forceinline__ float h_bits(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)u)); }
// A normal x > 0 as 2^e r with r in [1, 2): p2 = 2^e, returns r (else p2 = x, r = 1).
__device__ __forceinline__ float split_pow2(float x, float& p2) {
  const uint32_t b = __float_as_uint(x);
  p2 = b >> 23 ? __uint_as_float(b & 0x7f800000u) : x;
  return b >> 23 ? __uint_as_float((b & 0x7fffffu) | 0x3f800000u) : 1.f;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 .. 127

// Terms of non-finite V elements, which the products leave out (out of line: hardly ever taken).
// Outputs: rows r0 .. r0 + n - 1 of head h, this warp's row `i` and every column.
template <typename T>
__device__ __noinline__ void fix_outputs(const LinAttnArgs& a, const float* wv, int64_t r0, int i, int h) {
  const T* q = (const T*)a.q + (r0 + i) * a.q_stride + h * a.dk;
  T* out = (T*)a.out + ((r0 + i) * a.H + h) * a.dv;
  for (int j = 0; j <= i; ++j) {
    const T* v = (const T*)a.v + (r0 + j) * a.v_stride + h * a.dv;
    const T* k = (const T*)a.k + (r0 + j) * a.k_stride + h * a.dk;
    float z = 0.f;
    bool have = false;
    for (int e = 0; e < a.dv; ++e) {
      const float x = ld_f(v + e);
      if (isfinite(x)) continue;
      if (!have) {
        for (int d = 0; d < a.dk; ++d) z += ld_f(q + d) * ld_f(k + d);
        z *= a.scale * wv[C - 1 - (i - j)];
        have = true;
      }
      st_f(out + e, ld_f(out + e) + z * x);
    }
  }
}
// State: value row dv, columns col .. col + ncol - 1 of head h at TMEM address tS, which hold 2^b
// times the state after rows r0 .. r0 + n - 1.
template <typename T>
__device__ __noinline__ void fix_state(const LinAttnArgs& a, const float* wv, int64_t r0, int n, int h, int dv, int col,
                                       int ncol, uint32_t tS, float scale) {
  for (int b = 0; b < ncol; b += 32) {
    uint32_t u[32];
    __syncwarp();
    tld32(tS + b, u);
    ld_wait();
    pin32(u);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      const float v = ld_f((const T*)a.v + (r0 + t) * a.v_stride + h * a.dv + dv);
      if (isfinite(v)) continue;
      const T* k = (const T*)a.k + (r0 + t) * a.k_stride + h * a.dk + col + b;
      const float w = wv[C - n + t] * scale;   // lam^(n-1-t)
#pragma unroll
      for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) + w * v * ld_f(k + e));
    }
    __syncwarp();
    tst32(tS + b, u);
    st_wait();
  }
}

// OUT: outputs and final states from the segments' start states. !OUT: the segments' own
// contributions to the state into the workspace (all segments but each sequence's last).
template <typename T, int DK, int DV, bool OUT>
__global__ void __launch_bounds__(NTHREADS, 1)
    chunk_kernel(const __grid_constant__ Tab tab, const __grid_constant__ CUtensorMap mapQ,
                 const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const __grid_constant__ CUtensorMap mapO, const __grid_constant__ CUtensorMap mapIn,
                 const __grid_constant__ CUtensorMap mapWs, const __grid_constant__ CUtensorMap mapFin,
                 const __grid_constant__ LinAttnArgs a) {
  using L = Lay<DK, DV>;
  constexpr bool F16 = std::is_same<T, f16>::value;
  constexpr uint32_t BF = F16 ? 0 : 1;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = (uint64_t*)(sm + L::BAR);
  uint64_t* full = bars;                       // [3 of Q, K, V][2 stages] the tile has landed
  uint64_t* empty = bars + 6;                  // [3][2] its slot may be filled again
  uint64_t* clean = bars + 12;                 // [2] K and V: rows past the end and non-finite V are zeros
  uint64_t* p_full = bars + 14;                // Q K^T is in TMEM
  uint64_t* p_ready = bars + 15;               // weights and scaled Q are in TMEM
  uint64_t* s_ready = bars + 16;               // the state's copy is in shared memory, its decay applied
  uint64_t* v_ready = bars + 23;               // [2] the decayed values are in TMEM, V has been read for them
                                               // (two: the row warps may see one a chunk late)
  uint64_t* o_free = bars + 17;                // the outputs have left TMEM
  uint64_t* o_full = bars + 18;                // outputs are in TMEM
  uint64_t* ds_done = bars + 19;               // the state holds this chunk
  uint64_t* smax = bars + 20;                  // the start state's maximum over the warps is known (f16)
  uint64_t* mma_idle = bars + 21;              // [2]
  uint64_t* in_full = bars + 26;               // the start state is in shared memory
  uint64_t* in_free = bars + 27;               // it has been taken from there
  uint64_t* k_known = bars + 25;               // the exponents of K's rows are known (f16)
  uint64_t* p_read = bars + 28;                // Q K^T has left TMEM (bf16)
  uint64_t* r_known = bars + 29;               // [4 quadrants] both halves of its rows' largest weights are known (f16)
  uint32_t* tmem_slot = (uint32_t*)(bars + L::NBAR);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* v_flag = (volatile int*)(tmem_slot + 2);   // V has held a non-finite element
  // f16: powers of two from the magnitudes. Rows' bytes are exponents e, magnitudes below 2^e (-128: zeros).
  // What orders a slot's next write behind its last read:
  // v_exp: written for chunk c + 2 behind o_full(c), so behind p_ready(c), which the row warps arrive at after
  //   their read of chunk c's, and behind ds_done(c), so behind the value rows' own reads up to v_ready(c).
  // k_exp: written for chunk c + 2 behind p_full(c + 1), so behind the outputs of c and the row warps' p_ready(c).
  // w_exp: read up to p_ready(c), written for chunk c + 1 behind p_full(c + 1), so behind the outputs of c.
  // c_exp: the output warps read chunk c's up to o_free(c), which the outputs of c + 1 wait for; written for
  //   chunk c + 2 behind p_full(c + 2), so behind those.
  // bnd: chunk c's is read by the value rows up to s_ready(c); written for chunk c + 2 behind p_full(c + 1), so
  //   behind the outputs of c, which wait for s_ready(c).
  // wmax: written once. v_flag: only ever set.
  volatile float* wmax = (volatile float*)(tmem_slot + 3);   // [8] max |start state| per warp
  volatile float* bnd = (volatile float*)(tmem_slot + 11);   // [2] bound on the state before a chunk, by chunk parity
  volatile signed char* c_exp = (volatile signed char*)(tmem_slot + 13);   // [2][128] c of the rows, by chunk parity
  volatile signed char* w_exp = c_exp + 2 * C;             // [2 halves][128] the rows' weights, less 2
  volatile signed char* k_exp = w_exp + 2 * C;             // [2 parities][2 halves][128] the rows of K
  volatile signed char* v_exp = k_exp + 4 * C;             // [2][2][128] the rows of V
  float* wv = reinterpret_cast<float*>(sm + L::WV);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  // this CTA's segment
  const int h = blockIdx.x % a.H, seg = blockIdx.x / a.H;
  const bool is_full = seg < tab.fullcum[tab.n];
  const int s = is_full ? find(tab.fullcum, tab.n, seg) : find(tab.tailcum, tab.n, seg - tab.fullcum[tab.n]);
  const int n_full = tab.fullcum[s + 1] - tab.fullcum[s];
  const int k_seg = is_full ? seg - tab.fullcum[s] : n_full;   // segment of the sequence
  const bool last = k_seg + 1 == n_full + (tab.tailcum[s + 1] - tab.tailcum[s]);
  if (!OUT && last) {                          // (nothing needs its contribution)
    wait_prerequisites();
    allow_dependents();
    return;
  }
  const int len = tab.len[s], beg = k_seg * tab.seg_rows, end = min(len, beg + tab.seg_rows);
  const int nch = (end - beg + C - 1) / C;     // chunks (0 for an empty sequence)
  const int64_t row0 = (int64_t)tab.row0[s] + beg;
  const int ws_slot = tab.ws_seg[s] + k_seg;   // (of a sequence with several segments)
  // where the start state is, if there is one: as tiles of 32 floats x 32 value rows, copied into the
  // second stage's slots before that stage is used
  const bool from_ws = tab.ws_seg[s] >= 0;
  const bool has_start = OUT && (from_ws || a.S_in != nullptr);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&empty[i], F16 ? 8 : 1);       // Q: the row warps have read it (bf16: the outputs' products)
      mbar_init(&empty[2 + i], OUT ? 2 : 1);   // K: the products of the weights, and of the state
      mbar_init(&empty[4 + i], OUT ? 4 : 1);   // V: the outputs, staged there (!OUT: the state's products)
      mbar_init(&clean[i], 8);
      mbar_init(&v_ready[i], 8);
      mbar_init(&mma_idle[i], 1);
    }
    mbar_init(p_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(s_ready, 8);
    mbar_init(o_free, 4);
    mbar_init(o_full, 1);
    mbar_init(ds_done, 1);
    mbar_init(smax, 8);
    mbar_init(k_known, 8);
    mbar_init(in_full, 1);
    mbar_init(in_free, 8);
    mbar_init(p_read, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&r_known[i], 2);
    *abort_flag = 0;
    *v_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<TMEM_COLS>(tmem_slot);
  // The contributions' launch lets the next ones begin when the call's inputs are there. So the pass over
  // the chunks behind it (split) waits for its start state only, and loads its first chunk meanwhile (1024 x
  // 16 heads: 23.6 us without, 21.8 with).
  const bool late = OUT && tab.split;
  if (OUT) allow_dependents();
  if (!late) wait_prerequisites();
  if (!OUT) allow_dependents();
  auto settle = [&]() {                        // (before a bounded wait for what the start state leads to)
    if (late) wait_prerequisites();
  };
  const float l2 = log2_decay(a.log_decay[h]);
  if (threadIdx.x <= C) {
    const int d = threadIdx.x, tail = (end - beg) % C;
    wv[C - 1 - d] = exp2f(l2 * (float)d);
    if (d < C) wv[C + d] = d < tail ? exp2f(l2 * (float)(tail - 1 - d)) : 0.f;
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wwait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_given_up) ? 1 : 0) != 0;
  };
  // f16: the larger exponent of both halves, rows 4 lane .. + 3; those rows' weights lam^(n-1-t)
  auto exps4 = [&](volatile signed char* e, int* x) {
    const int a = *reinterpret_cast<volatile int*>(e + 4 * lane);
    const int b = *reinterpret_cast<volatile int*>(e + C + 4 * lane);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = max((int)(signed char)(a >> 8 * k), (int)(signed char)(b >> 8 * k));
  };
  auto weights4 = [&](int n, float* w) {
    const float4 v = *reinterpret_cast<const float4*>(wv + (n == C ? 0 : C) + 4 * lane);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  };
  auto start_bound = [&]() {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x = fmaxf(x, wmax[k]);
    return x;
  };
  // the state's scale exponent a
  auto scale_exp = [](float bound) { return bound > 0.f ? max(-114, min(100, 14 - exp_above(bound))) : 100; };
  auto pw = [&](int d) { return wv[C - 1 - d]; };   // lam^d, d = 0 .. 128
  auto arrive = [&](uint64_t* bar) {           // once per warp, after what it wrote
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == 0) {
    // ---- TMA producer
    if (lane == 0) {
      uint32_t fills = 0;                      // per slot: begun (bit i), parity of the last fill (bit 8 + i)
      bool ok = true;
      bool started = false;
      auto start = [&]() {
        settle();
        if (!has_start) return;
        started = true;
        mbar_expect_tx(in_full, DV * DK * 4);
        for (int b = 0; b < DK / 32; ++b)
          for (int y = 0; y < DV; y += 32)
            tma4(sm + L::STAGE + b * (DV * 128) + y * 128, from_ws ? &mapWs : &mapIn, in_full, 32 * b, y, h,
                 from_ws ? ws_slot : (a.s_in_stride ? tab.seq0 + s : 0));
      };
      if (nch == 0) start();
      for (int c = 0; c < nch && ok; ++c) {
        if (c == 1 && has_start) ok = mbar_wait(in_free, 0, abort_flag, &g_given_up);
        if (!ok) break;
        const int st = c & 1, r = (int)(row0 + c * C);
        uint8_t* base = sm + st * L::STAGE;
        auto load = [&](int which, const CUtensorMap* map, uint8_t* dst, int boxes, int bytes) {
          const int slot = 2 * which + st;
          ok = ok && mbar_wait(&empty[slot], ((c >> 1) & 1) ^ 1, abort_flag, &g_given_up);
          if (!ok) return;
          mbar_expect_tx(&full[slot], bytes);
          for (int b = 0; b < boxes; ++b) tma3(dst + b * C * 128, map, &full[slot], 64 * b, h, r);
          fills = (fills & ~(1u << (8 + slot))) | 1u << slot | (uint32_t)((c >> 1) & 1) << (8 + slot);
        };
        if (OUT) load(0, &mapQ, base, DK / 64, L::QB);
        load(1, &mapK, base + L::QB, DK / 64, L::QB);
        load(2, &mapV, base + 2 * L::QB, DV / 64, L::VB);
        if (c == 0) start();
      }
      if (*abort_flag && started) mbar_drain(in_full, 0);
      if (*abort_flag)                         // copies in flight land before the CTA leaves
        for (int i = 0; i < 6; ++i)
          if ((fills >> i) & 1) mbar_drain(&full[i], (fills >> (8 + i)) & 1);
    }
  } else if (warp == 1) {
    // ---- MMA issue: weights and outputs
    if constexpr (OUT) {
      const bool leader = elect_one();
      constexpr uint32_t ID_P = idesc_f16(C, BF, 0, 0), ID_QS = idesc_f16(DV, BF, 0, 0),
                         ID_PV = idesc_f16(DV, BF, 0, 1);
      for (int c = 0; c < nch; ++c) {
        const int st = c & 1;
        const uint32_t ph = c & 1, sph = (c >> 1) & 1;
        const uint32_t base = smem_u32(sm + st * L::STAGE);
        if (!wwait(&full[st], sph) || !wwait(&full[2 + st], sph)) break;
        if (!F16 && c > 0 && !wwait(ds_done, (c - 1) & 1)) break;   // (the third parts in these columns have been read)
        fence_after();
        if (leader) {                          // Q K^T (in order behind the products that read these columns)
          const uint64_t qd = desc_sw128(base, 16), kd = desc_sw128(base + L::QB, 16);
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * (C * 128) + (kk & 3) * 32) >> 4);
            mma_ss(tmem + T_P, qd + off, kd + off, ID_P, kk > 0 ? 1u : 0u);
          }
          commit(p_full);
          commit(&empty[2 + st]);
        }
        __syncwarp();
        if (c == 0) settle();
        if (!wwait(&clean[st], sph) || !wwait(s_ready, ph) || !wwait(p_ready, ph)) break;
        if (c > 0 && !wwait(o_free, (c - 1) & 1)) break;
        fence_after();
        if (leader) {                          // O = (scaled Q) S^T + weights V
          const uint64_t sd = desc_sw128(smem_u32(sm + L::S16), 16), vd = desc_sw128(base + 2 * L::QB, C * 128);
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint64_t so = sd + (uint64_t)(((kk >> 2) * (DV * 128) + (kk & 3) * 32) >> 4);
            if constexpr (F16) {
              const int q = kk < DK / 32 ? 32 + kk * 8 : 96 + (kk - DK / 32) * 8;
              mma_ts(tmem + T_O, tmem + T_P + q, so, ID_QS, kk > 0 ? 1u : 0u);
            } else {
              const uint64_t qo = desc_sw128(base, 16) + (uint64_t)(((kk >> 2) * (C * 128) + (kk & 3) * 32) >> 4);
              mma_ss(tmem + T_O, qo, so, ID_QS, kk > 0 ? 1u : 0u);
            }
          }
          if (!F16) commit(&empty[st]);
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_ts(tmem + T_O, tmem + T_P + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8),
                   vd + (uint64_t)(kk * 16 * 128 >> 4), ID_PV, 1u);
          commit(o_full);
        }
        __syncwarp();
      }
      if (leader) {
        commit(&mma_idle[0]);
        mbar_drain(&mma_idle[0], 0);           // every MMA issued above has completed
      }
    }
  } else if (warp == 18) {
    // ---- MMA issue: S += (decayed V)^T K, high and low parts
    const bool leader = elect_one();
    constexpr uint32_t ID_S = idesc_f16(DK, BF, 0, 1);
    settle();
    for (int c = 0; c < nch; ++c) {
      const int st = c & 1;
      if (!wwait(&full[2 + st], (c >> 1) & 1) || !wwait(&v_ready[st], (c >> 1) & 1)) break;
      fence_after();
      if (leader) {
        const uint64_t kd = desc_sw128(smem_u32(sm + st * L::STAGE + L::QB), C * 128);
        // (small parts first: the tensor cores' sums lose less)
        if constexpr (!F16) {
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_ts(tmem + T_S, tmem + T_P + (kk < 4 ? 32 + kk * 8 : 96 + (kk - 4) * 8),
                   kd + (uint64_t)(kk * 16 * 128 >> 4), ID_S, OUT || c > 0 || kk > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          mma_ts(tmem + T_S, tmem + T_VL + kk * 8, kd + (uint64_t)(kk * 16 * 128 >> 4), ID_S,
                 !F16 || OUT || c > 0 || kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          mma_ts(tmem + T_S, tmem + T_VH + kk * 8, kd + (uint64_t)(kk * 16 * 128 >> 4), ID_S, 1u);
        commit(ds_done);
        commit(&empty[2 + st]);
        if (!OUT) commit(&empty[4 + st]);
      }
      __syncwarp();
    }
    if (leader) {
      commit(&mma_idle[1]);
      mbar_drain(&mma_idle[1], 0);
    }
  } else if (warp < 10) {
    // ---- rows of the chunk: two threads per row i, each half of its weights (columns 64 half ..), of
    // its scaled Q. `scale` enters with the outputs
    if constexpr (OUT) {
      const int quad = warp & 3, half = (warp - 2) >> 2, i = quad * 32 + lane;
      const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
      constexpr int HQ = DK / 2;               // this half's Q elements
      const uint32_t tP = tmem + lane_off + T_P + half * 64;
      float qs;                                // lam^(i+1) = qs r: Q takes the power of two, the outputs r
      const float rinv = 1.f / split_pow2(pw(i + 1), qs);
      float bound = 0.f;                       // at least every finite |state element| (f16)
      if (F16) settle();
      if (F16 && nch > 0 && wwait(smax, 0)) bound = start_bound();
      for (int c = 0; c < nch; ++c) {
        const int st = c & 1;
        const uint32_t ph = c & 1, sph = (c >> 1) & 1;
        const uint8_t* qrow = sm + st * L::STAGE + i * 128;
        auto q16 = [&](int q) {                // 16-byte chunk q of the Q row
          return *reinterpret_cast<const uint4*>(qrow + (q >> 3) * (C * 128) + (((q & 7) ^ (i & 7)) << 4));
        };
        if (!wwait(&full[st], sph)) break;
        float fp = rinv, fq = qs;
        uint32_t qm = 0;                       // max |Q| of the row (f16)
        float next = 0.f;                      // the bound after this chunk
        if constexpr (F16) {
          uint32_t m = 0, mk = 0;
#pragma unroll 4
          for (int q = 0; q < DK / 8; ++q) {
            const uint4 v = q16(q);
            m = absmax2(T(), m, absmax2(T(), absmax2(T(), v.x, v.y), absmax2(T(), v.z, v.w)));
          }
          qm = max(m & 0xffffu, m >> 16);
          if (qm >= 0x7c00u) qm = 0;           // (a row with a non-finite element: no scale makes its outputs finite)
          if (!wwait(&full[2 + st], sph)) break;
          if (c + 1 < nch) {                   // (the last chunk: nothing follows)
            // this half of row i of K; non-finite elements aside
            const uint8_t* krow = sm + st * L::STAGE + L::QB + i * 128;
            auto k16 = [&](int q) {
              q += half * (DK / 16);
              return *reinterpret_cast<const uint4*>(krow + (q >> 3) * (C * 128) + (((q & 7) ^ (i & 7)) << 4));
            };
#pragma unroll 4
            for (int q = 0; q < DK / 16; ++q) {
              const uint4 v = k16(q);
              mk = absmax2(T(), mk, absmax2(T(), absmax2(T(), v.x, v.y), absmax2(T(), v.z, v.w)));
            }
            if (max(mk & 0xffffu, mk >> 16) >= 0x7c00u) {
              mk = 0;
#pragma unroll 1
              for (int q = 0; q < DK / 16; ++q) {
                const uint4 v = k16(q);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  mk = absmax2(T(), mk, (nonfinite(T(), w[e] & 0xffffu) ? 0u : w[e] & 0x7fffu) |
                                            (nonfinite(T(), w[e] >> 16) ? 0u : w[e] & 0x7fff0000u));
              }
            }
            mk = max(mk & 0xffffu, mk >> 16);
            const bool in = i < end - beg - c * C;
            k_exp[(ph * 2 + half) * C + i] = (signed char)(mk > 0 && in ? exp_above(h_bits(mk)) : -128);
            arrive(k_known);
            // the state after this chunk: lam^n S and the terms, row by row
            if (!wwait(&clean[st], sph) || !wwait(k_known, ph)) break;
            const int n = min(C, end - beg - c * C);
            int ke[4], ve[4];
            float w[4], add = 0.f;
            exps4(k_exp + ph * 2 * C, ke);
            exps4(v_exp + ph * 2 * C, ve);
            weights4(n, w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (ke[k] + ve[k] > -100) add += w[k] * pow2f(ke[k] + ve[k]);
            next = 1.00001f * (bound * pw(n)) + 1.0001f * warp_sum(add);
          }
        }
        if (!wwait(p_full, ph)) break;
        fence_after();
        if constexpr (F16) {                   // c of the row, from its own weights: fp32, decayed, in place
          float mx = 0.f;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            const int b = 64 * half + 32 * k;
            if (b > quad * 32) break;
            uint32_t u[32];
            __syncwarp();
            tld32(tP + 32 * k, u);
            ld_wait();
            pin32(u);
            const float* w = wv + C - 1 - i + b;   // lam^(i-b-e) at w[e] (past the diagonal: not used)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = b + e <= i ? __uint_as_float(u[e]) * w[e] : 0.f;
              mx = fmaxf(mx, fabsf(x));
              u[e] = __float_as_uint(x);
            }
            tst32(tP + 32 * k, u);
          }
          st_wait();
          w_exp[half * C + i] = (signed char)(mx > 0.f ? exp_above(mx) - 2 : -128);   // (-125 .. 129, - 2)
          arrive(&r_known[quad]);
          if (!wwait(&r_known[quad], ph)) break;
          const int we = max(w_exp[i], w_exp[C + i]), sa = scale_exp(bound);
          int cexp = 100;
          if (we > -128) cexp = min(cexp, 12 - we);
          // (q 2^e, where qs = 2^e or, below the normal numbers, less than 2^-126)
          const int eq = exp_above(h_bits(qm)) + max((int)(__float_as_uint(qs) >> 23), 1) - 127;
          if (qm > 0 && qs > 0.f && sa < 100) cexp = min(cexp, sa + 14 - eq);
          cexp = max(cexp, -120);
          fp = pow2f(cexp) * rinv;
          const int qe = cexp - sa;            // |q| qs 2^qe < 2^14, or the state is zero
          fq = qe < -126 ? 0.f : qe > 126 ? qs * pow2f(126) * pow2f(qe - 126) : qs * pow2f(qe);
          if (half == 0) c_exp[ph * C + i] = (signed char)cexp;
          bound = next;
          if (warp == 2 && lane == 0) bnd[ph ^ 1] = next;
        }
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          // 32 weights of V: lam^(i-j) q_i.k_j, 0 for j > i; 16-bit in place, behind what is still to be read
          const int b = 64 * half + 32 * k;
          uint32_t p[16];
          if (b > quad * 32) {                 // behind every row of this warp
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0;
          } else {
            uint32_t u[32];
            __syncwarp();
            tld32(tP + 32 * k, u);
            ld_wait();
            pin32(u);
            if constexpr (F16) {
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                p[e / 2] = pack(T(), __uint_as_float(u[e]) * fp, __uint_as_float(u[e + 1]) * fp);
            } else {
              const float* w = wv + C - 1 - i + b;   // lam^(i-b-e) at w[e] (past the diagonal: not used)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float x0 = __uint_as_float(u[e]) * (w[e] * fp);
                const float x1 = __uint_as_float(u[e + 1]) * (w[e + 1] * fp);
                p[e / 2] = pack(T(), b + e <= i ? x0 : 0.f, b + e + 1 <= i ? x1 : 0.f);
              }
            }
          }
          __syncwarp();
          tst16(tP + 16 * k, p);
        }
        if constexpr (!F16) {
          fence_before();
          arrive(p_read);
        }
#pragma unroll 1
        for (int k = 0; k < HQ / 32; ++k) {    // scaled Q
          uint32_t u[16];
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const uint4 v = q16(half * (HQ / 8) + 4 * k + k4);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack(T(), w[e]);
              u[4 * k4 + e] = pack(T(), f.x * fq, f.y * fq);
            }
          }
          if constexpr (F16) {
            tst16(tP + 32 + 16 * k, u);
          } else {                             // in place
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              const int q = half * (HQ / 8) + 4 * k + k4;
              *reinterpret_cast<uint4*>(const_cast<uint8_t*>(qrow) + (q >> 3) * (C * 128) + (((q & 7) ^ (i & 7)) << 4)) =
                  make_uint4(u[4 * k4], u[4 * k4 + 1], u[4 * k4 + 2], u[4 * k4 + 3]);
            }
          }
        }
        st_wait();
        if (!F16) fence_async_smem();
        fence_before();
        arrive(p_ready);
        if (F16 && lane == 0) mbar_arrive(&empty[st]);
        if (!F16 && c == 0) settle();
      }
    }
  } else if (warp >= 19) {
    // ---- outputs: thread = row i; scaled, staged in the V tile (which nothing else reads any more),
    // stored in whole rows
    if constexpr (OUT) {
      const int quad = warp & 3, i = quad * 32 + lane;
      const uint32_t tO = tmem + ((uint32_t)(quad * 32) << 16) + T_O;
      settle();
      float p2;
      const float fr = a.scale * split_pow2(pw(i + 1), p2);
      for (int c = 0; c < nch; ++c) {
        const int st = c & 1, n = min(C, end - beg - c * C);
        if (!wwait(o_full, c & 1) || !wwait(&v_ready[st], (c >> 1) & 1)) break;
        fence_after();
        const float f = F16 ? fr * pow2f(-c_exp[(c & 1) * C + i]) : fr;
        const uint64_t f2 = pack2(f, f);
        const bool fix = *v_flag;
        uint8_t* stage = sm + st * L::STAGE + 2 * L::QB;
#pragma unroll 1
        for (int b = 0; b < DV; b += 32) {
          uint32_t u[32];
          __syncwarp();
          tld32(tO + b, u);
          ld_wait();
          pin32(u);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t x = mul2(pack2u(u[e + 2 * k], u[e + 2 * k + 1]), f2);
              o[k] = pack(T(), lo2(x), hi2(x));
            }
            const int q = (b + e) / 8;         // (the layout of a TMA tile: boxes of 64 columns, swizzled)
            *reinterpret_cast<uint4*>(stage + (q >> 3) * (C * 128) + i * 128 + (((q & 7) ^ (i & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_before();
        fence_async_smem();                    // (read by the TMA store, and the slot's next fill is a TMA write)
        arrive(o_free);                        // (also orders the stage's writes within the warp)
        if (quad * 32 + 32 <= n) {             // 32 whole rows
          if (lane == 0) {
            for (int b = 0; b < DV / 64; ++b)
              tma3_store(&mapO, stage + b * (C * 128) + quad * 32 * 128, 64 * b, h, (int)(row0 + c * C + quad * 32));
            tma_store_commit();
            tma_store_read_wait();
          }
        } else {
          constexpr int CH = DV / 8;           // 16-byte chunks of a row
#pragma unroll 1
          for (int k = 0; k < CH; ++k) {
            const int e = k * 32 + lane, r = quad * 32 + e / CH, q = e % CH;
            if (r < n)
              *reinterpret_cast<uint4*>((T*)a.out + ((row0 + c * C + r) * a.H + h) * DV + q * 8) =
                  *reinterpret_cast<const uint4*>(stage + (q >> 3) * (C * 128) + r * 128 + (((q & 7) ^ (r & 7)) << 4));
          }
          fence_async_smem();
        }
        if (fix) {
          if (lane == 0) tma_store_wait();
          __syncwarp();
          if (i < n) fix_outputs<T>(a, wv, row0 + c * C, i, h);
        }
        arrive(&empty[4 + st]);
      }
      if (lane == 0) tma_store_wait();         // the stores are complete before the CTA leaves
    }
  } else {
    // ---- value rows: two threads per row dv of the state (64 value rows: twice over the 128 lanes),
    // each half of its columns, and half of the chunk's rows of the decayed values
    const int wi = warp - 10, quad = warp & 3, half = wi >> 2, r = quad * 32 + lane, dv = r % DV;
    constexpr int HK = DK / 2;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + T_S + half * HK;
    const uint32_t tVH = tmem + lane_off + T_VH + half * 32, tVL = tmem + lane_off + T_VL + half * 32;
    bool ok = true;
    int bexp = 0;                              // b: the state in TMEM is 2^b times the state (f16)
    // adds chunk c's terms of non-finite V elements to this thread's state columns
    auto fix = [&](int c) {
      if (*v_flag)
        fix_state<T>(a, wv, row0 + c * C, min(C, end - beg - c * C), h, dv, half * HK, HK, tS,
                     F16 ? pow2f(bexp) : 1.f);
    };
    // 32 columns of this thread's state row, unscaled
    auto state32 = [&](int b, float* x) {
      uint32_t u[32];
      __syncwarp();
      tld32(tS + b, u);
      ld_wait();
      pin32(u);
      const float f = F16 ? pow2f(-bexp) : 1.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = F16 ? __uint_as_float(u[e]) * f : __uint_as_float(u[e]);
    };
    float bound = 0.f;                         // at least every finite |state element| (f16)
    // rows past the end to zeros (K and V), non-finite V elements to zero; f16: the exponents of V's rows. A
    // thread takes DV / 16 chunks of 16 bytes of V: half of row r (bf16: in memory order)
    auto cleaning = [&](int c) {
      const int st = c & 1, n = min(C, end - beg - c * C);
      const uint32_t sph = (c >> 1) & 1;
      uint8_t* kt = sm + st * L::STAGE + L::QB;
      uint8_t* vt = kt + L::QB;
      constexpr int KC = DK / 8, VQ = DV / 16;
      const int tid = wi * 32 + lane;
      auto v16 = [&](int q) {
        const int x = half * VQ + q;
        return reinterpret_cast<uint4*>(F16 ? vt + (x >> 3) * (C * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4)
                                            : vt + (q * 256 + tid) * 16);
      };
      auto past = [&](int q) { return (F16 ? r : ((q * 256 + tid) >> 3) % C) >= n; };
      if (!wwait(&full[2 + st], sph) || !wwait(&full[4 + st], sph)) return false;
      bool bad = false, wrote = n < C;
      uint32_t vm = 0;
      {
        uint4 v[VQ];
#pragma unroll
        for (int q = 0; q < VQ; ++q) v[q] = *v16(q);
#pragma unroll
        for (int q = 0; q < VQ; ++q) {
          const uint32_t x = absmax2(T(), absmax2(T(), v[q].x, v[q].y), absmax2(T(), v[q].z, v[q].w));
          if (!past(q)) vm = absmax2(T(), vm, x);
          else *v16(q) = make_uint4(0, 0, 0, 0);
        }
      }
      if (max(vm & 0xffffu, vm >> 16) >= (F16 ? 0x7c00u : 0x7f80u)) {   // some element is to be replaced
        vm = 0;
#pragma unroll 1
        for (int q = 0; q < VQ; ++q) {
          uint32_t* at = reinterpret_cast<uint32_t*>(v16(q));
          if (past(q)) continue;
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            uint32_t w = at[e];
            const bool lo = nonfinite(T(), w & 0xffffu), hi = nonfinite(T(), w >> 16);
            bad |= lo || hi;
            if (lo) w &= 0xffff0000u;
            if (hi) w &= 0xffffu;
            at[e] = w;
            vm = absmax2(T(), vm, w);
          }
        }
        wrote = true;
      }
      if (n < C)
        for (int e = tid; e < (C - n) * KC; e += 256) {
          const int t = n + e / KC, q = e % KC;
          *reinterpret_cast<uint4*>(kt + (q >> 3) * (C * 128) + t * 128 + ((q & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
      if (bad) *v_flag = 1;
      if constexpr (F16) {
        vm = max(vm & 0xffffu, vm >> 16);
        v_exp[(st * 2 + half) * C + r] = (signed char)(vm > 0 ? exp_above(h_bits(vm)) : -128);
      }
      if (wrote) fence_async_smem();
      arrive(&clean[st]);
      return true;
    };
    // this thread's place for columns b + 4 e .. + 3 of a state row in shared memory (swizzled tiles)
    auto state_at = [&](uint8_t* base, int b, int e) {
      const int col = half * HK + b;
      return reinterpret_cast<float4*>(base + (col >> 5) * (DV * 128) + dv * 128 + ((e ^ (dv & 7)) << 4));
    };
    if (nch > 0) ok = cleaning(0);
    if constexpr (OUT) {
      // the start state into TMEM
      settle();
      if (ok && has_start) ok = wwait(in_full, 0);
#pragma unroll 1
      for (int b = 0; b < HK && ok; b += 32) {
        uint32_t u[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 v = has_start ? *state_at(sm + L::STAGE, b, e) : make_float4(0.f, 0.f, 0.f, 0.f);
          u[4 * e] = __float_as_uint(v.x);
          u[4 * e + 1] = __float_as_uint(v.y);
          u[4 * e + 2] = __float_as_uint(v.z);
          u[4 * e + 3] = __float_as_uint(v.w);
        }
        if constexpr (F16) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = fabsf(__uint_as_float(u[e]));
            if (x < INFINITY) bound = fmaxf(bound, x);
          }
        }
        __syncwarp();
        tst32(tS + b, u);
      }
      st_wait();
      if (has_start) {
        fence_async_smem();                    // (the slots' next fill is a TMA write)
        arrive(in_free);
      }
      if constexpr (F16) {
        bound = warp_max(bound);
        if (lane == 0) wmax[wi] = bound;
        arrive(smax);
        if (ok) ok = wwait(smax, 0);
        bound = start_bound();
      }
    }
    for (int c = 0; c < nch && ok; ++c) {
      const int st = c & 1, n = min(C, end - beg - c * C);
      const uint32_t sph = (c >> 1) & 1;
      const uint8_t* vt = sm + st * L::STAGE + 2 * L::QB;
      if (!wwait(&clean[st], sph)) { ok = false; break; }   // (all warps' shares)
      if (c > 0 && !wwait(ds_done, (c - 1) & 1)) { ok = false; break; }
      if (OUT && c > 0 && !wwait(o_full, (c - 1) & 1)) { ok = false; break; }   // (its state copy has been read)
      int bnew = 0, sa = 0;
      if constexpr (F16) {                     // decayed values below 2^14, and the scaled state finite
        if (OUT && c > 0) bound = bnd[st];
        int ve[4];
        float w[4], x = 0.f;
        exps4(v_exp + st * 2 * C, ve);
        weights4(n, w);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (ve[k] > -128) x = fmaxf(x, w[k] * pow2f(ve[k]));
        x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
        if (x > 0.f) bnew = min(60, 14 - exp_above(x));
        if (bound > 0.f) bnew = min(bnew, 120 - exp_above(bound));
        sa = scale_exp(bound);
      }
      fence_after();
      // state: operand copy (scaled for f16), then decayed in place
      if (OUT || c > 0) {
        if (c > 0) fix(c - 1);
        const float f = F16 ? pow2f(sa) : 1.f;
        const float ds = F16 ? pw(n) * pow2f(bnew) : pw(n);
#pragma unroll 1
        for (int b = 0; b < HK; b += 32) {
          float x[32];
          state32(b, x);
          if (OUT && r < DV) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* y = x + 8 * k;
              const int q = (half * HK + b) / 8 + k;
              *reinterpret_cast<uint4*>(sm + L::S16 + (q >> 3) * (DV * 128) + r * 128 + (((q & 7) ^ (r & 7)) << 4)) =
                  make_uint4(pack(T(), y[0] * f, y[1] * f), pack(T(), y[2] * f, y[3] * f),
                             pack(T(), y[4] * f, y[5] * f), pack(T(), y[6] * f, y[7] * f));
            }
          }
          uint32_t u[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(x[e] * ds);
          __syncwarp();
          tst32(tS + b, u);
        }
        if constexpr (OUT) {
          st_wait();
          fence_async_smem();
          fence_before();
          arrive(s_ready);
        }
      }
      bexp = bnew;
      // decayed values of rows 64 half .. +63, split: high part (nearest), low part (what it leaves)
      {
        const float sb = F16 ? pow2f(bnew) : 1.f;
        const uint8_t* col = vt + (dv >> 6) * (C * 128) + (dv & 7) * 2 + half * (64 * 128);
        const int ch = (dv & 63) >> 3;
        const float* w = wv + (n == C ? 0 : C) + half * 64;
        if (!F16 && OUT) {                     // (the weights' columns that the third parts take)
          if (!wwait(p_read, c & 1)) { ok = false; break; }
          fence_after();
        }
#pragma unroll 1
        for (int t0 = 0; t0 < 64; t0 += 32) {
          uint32_t hi[16], lo[16], third[16];
#pragma unroll
          for (int t = 0; t < 32; t += 4) {
            const float4 w4 = *reinterpret_cast<const float4*>(w + t0 + t);
            const float ww[4] = {w4.x, w4.y, w4.z, w4.w};
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const T v = *reinterpret_cast<const T*>(col + (t0 + t + e) * 128 + ((ch ^ ((t + e) & 7)) << 4));
              y[e] = ld_f(&v) * (F16 ? ww[e] * sb : ww[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint32_t hp = pack(T(), y[e], y[e + 1]);
              const float2 f = unpack(T(), hp);
              hi[(t + e) / 2] = hp;
              lo[(t + e) / 2] = pack(T(), y[e] - f.x, y[e + 1] - f.y);
              if constexpr (!F16) {
                const float2 g = unpack(T(), lo[(t + e) / 2]);
                third[(t + e) / 2] = pack(T(), y[e] - f.x - g.x, y[e + 1] - f.y - g.y);
              }
            }
          }
          tst16(tVH + t0 / 2, hi);
          tst16(tVL + t0 / 2, lo);
          if constexpr (!F16) tst16(tmem + lane_off + T_P + half * 64 + 32 + t0 / 2, third);
        }
      }
      st_wait();
      fence_before();
      arrive(&v_ready[st]);
      if (c + 1 < nch && !cleaning(c + 1)) { ok = false; break; }
    }
    // ---- the state after the segment
    // stored through the other stage's Q and K slots (nothing is loaded any more), 32 rows a warp
    const bool keep = OUT ? last && a.S_out != nullptr : true;
    if (ok && nch > 0) ok = wwait(ds_done, (nch - 1) & 1);
    fence_after();
    if (ok && nch > 0) fix(nch - 1);
    if (ok && keep) {
      uint8_t* stage = sm + (nch & 1) * L::STAGE;
#pragma unroll 1
      for (int b = 0; b < HK; b += 32) {
        float x[32];
        state32(b, x);
        if (r < DV)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *state_at(stage, b, e) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0 && quad * 32 < DV) {
        for (int b = 0; b < HK; b += 32)
          tma4_store(OUT ? &mapFin : &mapWs, stage + ((half * HK + b) >> 5) * (DV * 128) + quad * 32 * 128,
                     half * HK + b, quad * 32, h, OUT ? tab.seq0 + s : ws_slot);
        tma_store_commit();
        tma_store_wait();
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<TMEM_COLS>(tmem);
  }
}

// Start states: in each sequence of several segments, slot k of the workspace (segment k's own
// contribution) becomes the state before segment k (segment 0's is the initial state: the last
// segment may overwrite that one in place). One thread per four state elements; the serial part is one
// multiply-add a segment, its loads are issued ahead (eight segments of 16 heads: 6.5 us from cold caches,
// mostly latency).
__global__ void __launch_bounds__(256)
    scan_kernel(const __grid_constant__ Tab tab, const __grid_constant__ LinAttnArgs a) {
  allow_dependents();
  wait_prerequisites();
  const int s = blockIdx.y;
  if (tab.ws_seg[s] < 0) return;
  const int64_t per4 = (int64_t)a.H * a.dv * a.dk / 4, hd4 = (int64_t)a.dv * a.dk / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= per4) return;
  const float f = exp2f(log2_decay(a.log_decay[i / hd4]) * (float)tab.seg_rows);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.S_in)
    S = *reinterpret_cast<const float4*>(a.S_in + (int64_t)(tab.seq0 + s) * a.s_in_stride + 4 * i);
  const int n = tab.fullcum[s + 1] - tab.fullcum[s] + tab.tailcum[s + 1] - tab.tailcum[s];
  float4* w = reinterpret_cast<float4*>(a.ws) + (int64_t)tab.ws_seg[s] * per4 + i;
  constexpr int AHEAD = 8;                     // contributions loaded before they are joined
  for (int k0 = 0; k0 + 1 < n; k0 += AHEAD) {
    float4 b[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k0 + k + 1 < n) b[k] = w[(int64_t)(k0 + k) * per4];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k0 + k + 1 < n) {
        w[(int64_t)(k0 + k) * per4] = S;
        S.x = f * S.x + b[k].x;
        S.y = f * S.y + b[k].y;
        S.z = f * S.z + b[k].z;
        S.w = f * S.w + b[k].w;
      }
  }
  w[(int64_t)(n - 1) * per4] = S;
}

// One token per sequence. A block takes 32 value rows of one (sequence, head), a warp 8 of them:
// the state is read and written once, coalesced rows of dk floats. Bound by those bytes: 255 sequences x 32
// heads of 128 x 128 173 us, 6.2 TB/s; three sequences x 16 heads, reading only, 3.2 us, a launch.
constexpr int STEP_ROWS = 8;
template <typename T, int DK>
__global__ void __launch_bounds__(128)
    step_kernel(const LinAttnArgs a, int n) {
  constexpr int E = DK / 32;
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slices = a.dv / 32;
  const uint32_t b = blockIdx.x;
  const int slice = b % slices;
  const uint32_t sh = b / slices;
  const int h = sh % a.H;
  const int64_t s = sh / a.H;
  const int r0 = slice * 32 + warp * STEP_ROWS;
  const int64_t at = ((int64_t)h * a.dv + r0) * DK + lane * E, per = (int64_t)a.H * a.dv * DK;
  float S[STEP_ROWS][E], q[E], k[E];
#pragma unroll
  for (int i = 0; i < STEP_ROWS; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) S[i][e] = a.S_in ? a.S_in[s * a.s_in_stride + at + i * DK + e] : 0.f;
  const T* qp = (const T*)a.q + s * a.q_stride + h * DK + lane * E;
  const T* kp = (const T*)a.k + s * a.k_stride + h * DK + lane * E;
  const T* vp = (const T*)a.v + s * a.v_stride + h * a.dv + r0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = ld_f(qp + e) * a.scale;
    k[e] = ld_f(kp + e);
  }
  const float lam = decay(a.log_decay[h]);
#pragma unroll
  for (int i = 0; i < STEP_ROWS; ++i) {
    const float v = ld_f(vp + i);
    float o = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      S[i][e] = lam * S[i][e] + v * k[e];
      o += S[i][e] * q[e];
      if (a.S_out) a.S_out[s * per + at + i * DK + e] = S[i][e];
    }
    o = warp_sum(o);
    if (lane == 0) st_f((T*)a.out + (s * a.H + h) * a.dv + r0 + i, o);
  }
}

}  // namespace lin

cudaError_t linattn_gave_up_word(uint64_t** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), lin::g_given_up);
}

// Rows per segment (a multiple of the chunk) for a group of sequences: the count with the least
// estimated time in us. A CTA's cost is a fixed part and a part per chunk, as measured at 128 x 128 (3.1
// us a chunk on a few SMs, 4.0 when all of them read and write); the full segments fill the SMs in
// rounds, the shorter last ones go where SMs are free, and end half of one later than if they could be
// divided. Against the best of up to 26 forced lengths, over 10 calls from 500 rows to 16476: within 4 %.
static int seg_rows_for(const int* len, int n, int H, int dk, int dv, int num_sms) {
  int longest = 1;
  for (int s = 0; s < n; ++s) longest = std::max(longest, len[s]);
  const double area = (double)dk * dv / (128.0 * 128.0);
  const int max_ch = (int)(((int64_t)longest + lin::C - 1) / lin::C);
  int best_m = max_ch;
  double best = 1e300;
  for (int m = max_ch; m >= 1; m = m > 8 ? m - (m + 15) / 16 : m - 1) {
    const int64_t L = (int64_t)m * lin::C;
    // full segments, shorter last ones and their chunks, segments before a sequence's last, start states
    int64_t full = 0, tails = 0, tail_ch = 0, longest_tail = 0, inner = 0, slots = 0;
    for (int s = 0; s < n; ++s) {
      const int64_t f = len[s] / L, rest = len[s] - f * L, segs = f + (rest > 0 || len[s] == 0 ? 1 : 0);
      full += f * H;
      if (segs > f) {
        const int64_t ch = (rest + lin::C - 1) / lin::C;
        tails += H;
        tail_ch += ch * H;
        longest_tail = std::max(longest_tail, ch);
      }
      if (segs > 1) {
        slots += segs * H;
        inner += (segs - 1) * H;
      }
    }
    const double chunk = 3.1 + 0.9 * (double)std::min<int64_t>(full + tails, num_sms) / num_sms, fixed = 6.0;
    const double each = chunk * m + fixed;
    const double t0 = (double)(full / num_sms) * each, over = (double)(full % num_sms);
    double t = t0 + (over > 0 ? each : 0.0);
    if (tails) {
      const double rest = chunk * (double)tail_ch + fixed * (double)tails;
      t = std::max(t, t0 + chunk * (double)longest_tail + fixed);
      if (tails > num_sms - (int64_t)over) t = std::max(t, t0 + (over * each + rest) / num_sms + 0.5 * rest / (double)tails);
    }
    if (slots) t += (double)((inner + num_sms - 1) / num_sms) * (1.8 * m + 4.0) + 4.0 + (double)slots * area * 0.02;
    if (t < best) {
      best = t;
      best_m = m;
    }
  }
  return (int)std::min<int64_t>((int64_t)best_m * lin::C, INT_MAX - INT_MAX % lin::C);
}

// Fills `t` with sequences from `s` on; returns the first one not taken. *slots: start states that
// the group keeps in the workspace.
static int lin_group(lin::Tab& t, int s, int n_seq, const int* row0, const int* len, int H, int dk, int dv,
                     int num_sms, int64_t* slots) {
  t.seq0 = s;
  t.n = std::min(n_seq - s, lin::MAX_SEQ);
  t.seg_rows = seg_rows_for(len + s, t.n, H, dk, dv, num_sms);
  t.fullcum[0] = t.tailcum[0] = 0;
  *slots = 0;
  t.split = 0;
  for (int i = 0; i < t.n; ++i) {
    const int full = len[s + i] / t.seg_rows, tail = len[s + i] % t.seg_rows > 0 || len[s + i] == 0 ? 1 : 0;
    t.row0[i] = row0 ? row0[s + i] : 0;
    t.len[i] = len[s + i];
    t.fullcum[i + 1] = t.fullcum[i] + full;
    t.tailcum[i + 1] = t.tailcum[i] + tail;
    t.ws_seg[i] = full + tail > 1 ? (int)*slots : -1;
    if (full + tail > 1) *slots += full + tail, t.split = 1;
  }
  return s + t.n;
}

int64_t linattn_ws_bytes(int n_seq, const int* len, int H, int dk, int dv, int num_sms) {
  int64_t need = 0, slots;
  lin::Tab t;
  for (int s = 0; s < n_seq;) {
    s = lin_group(t, s, n_seq, nullptr, len, H, dk, dv, num_sms, &slots);
    need = std::max(need, slots * H * dk * dv * 4);
  }
  return need;
}

template <typename T, int DK, int DV>
static cudaError_t lin_launch(const LinAttnArgs& a, const lin::Tab& t, int64_t slots, const CUtensorMap* m,
                              cudaStream_t st) {
  using L = lin::Lay<DK, DV>;
  const dim3 grid((unsigned)((int64_t)(t.fullcum[t.n] + t.tailcum[t.n]) * a.H)), block(lin::NTHREADS);
  if (slots > 0) {
    CK_RET(cudaFuncSetAttribute(lin::chunk_kernel<T, DK, DV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::BYTES));
    CK_RET(launch_pdl(lin::chunk_kernel<T, DK, DV, false>, grid, block, L::BYTES, st, t, m[0], m[1], m[2], m[3],
                      m[4], m[5], m[6], a));
    const int64_t per4 = (int64_t)a.H * DK * DV / 4;
    CK_RET(launch_pdl(lin::scan_kernel, dim3((unsigned)((per4 + 255) / 256), t.n), dim3(256), 0, st, t, a));
  }
  CK_RET(cudaFuncSetAttribute(lin::chunk_kernel<T, DK, DV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
  return launch_pdl(lin::chunk_kernel<T, DK, DV, true>, grid, block, L::BYTES, st, t, m[0], m[1], m[2], m[3], m[4],
                    m[5], m[6], a);
}

cudaError_t launch_linattn(const LinAttnArgs& a, int n_seq, const int* row0, const int* len, int num_sms,
                           cudaStream_t st) {
  int64_t rows = 1;
  for (int s = 0; s < n_seq; ++s)
    if (len[s]) rows = std::max(rows, (int64_t)row0[s] + len[s]);
  CUtensorMap m[7] = {};                       // q, k, v, out; initial states, start states, final states
  const CUtensorMapDataType ty =
      a.dtype == ELEM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const void* ptr[4] = {a.q, a.k, a.v, a.out};
  const int d[4] = {a.dk, a.dk, a.dv, a.dv};
  const int64_t ld[4] = {a.q_stride, a.k_stride, a.v_stride, (int64_t)a.H * a.dv};
  for (int i = 0; i < 4; ++i) {
    const uint64_t dims[3] = {(uint64_t)d[i], (uint64_t)a.H, (uint64_t)rows};
    const uint64_t str[2] = {(uint64_t)d[i] * 2, (uint64_t)ld[i] * 2};
    const uint32_t box[3] = {64, 1, i < 3 ? (uint32_t)lin::C : 32u};
    if (!encode_tensor_map(&m[i], ty, 3, ptr[i], dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  auto state_map = [&](CUtensorMap* map, const void* base, int64_t n) {   // [n][H][dv][dk] fp32
    const uint64_t dims[4] = {(uint64_t)a.dk, (uint64_t)a.dv, (uint64_t)a.H, (uint64_t)n};
    const uint64_t str[3] = {(uint64_t)a.dk * 4, (uint64_t)a.dv * a.dk * 4, (uint64_t)a.H * a.dv * a.dk * 4};
    const uint32_t box[4] = {32, 32, 1, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (a.S_in && !state_map(&m[4], a.S_in, a.s_in_stride ? n_seq : 1)) return cudaErrorInvalidValue;
  if (a.S_out && !state_map(&m[6], a.S_out, n_seq)) return cudaErrorInvalidValue;
  lin::Tab t;
  for (int s = 0; s < n_seq;) {
    int64_t slots;
    s = lin_group(t, s, n_seq, row0, len, a.H, a.dk, a.dv, num_sms, &slots);
    if (((int64_t)t.fullcum[t.n] + t.tailcum[t.n]) * a.H > INT_MAX) return cudaErrorInvalidValue;
    if (slots > 0 && !state_map(&m[5], a.ws, slots)) return cudaErrorInvalidValue;
#define LIN_GO(T)                                                                                        \
  CK_RET(a.dk == 128 ? (a.dv == 128 ? lin_launch<T, 128, 128>(a, t, slots, m, st)                   \
                                    : lin_launch<T, 128, 64>(a, t, slots, m, st))                   \
                     : (a.dv == 128 ? lin_launch<T, 64, 128>(a, t, slots, m, st)                    \
                                    : lin_launch<T, 64, 64>(a, t, slots, m, st)))
    if (a.dtype == ELEM_F16) LIN_GO(f16);
    else LIN_GO(bf16);
#undef LIN_GO
  }
  return cudaSuccess;
}

cudaError_t launch_linattn_step(const LinAttnArgs& a, int n, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)n * a.H * (a.dv / 32))), block(128);
  if (a.dtype == ELEM_F16)
    return a.dk == 128 ? launch_pdl(lin::step_kernel<f16, 128>, grid, block, 0, st, a, n)
                       : launch_pdl(lin::step_kernel<f16, 64>, grid, block, 0, st, a, n);
  return a.dk == 128 ? launch_pdl(lin::step_kernel<bf16, 128>, grid, block, 0, st, a, n)
                     : launch_pdl(lin::step_kernel<bf16, 64>, grid, block, 0, st, a, n);
}

}  // namespace s1
