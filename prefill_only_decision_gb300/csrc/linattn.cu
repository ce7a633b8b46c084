// Linear attention with a decay per head: S_t = lam_h S_{t-1} + v_t k_t^T, o_t = scale S_t q_t,
// lam_h = exp(log_decay[h]). Prompts (launch_linattn) and single tokens (launch_linattn_step).
#include <algorithm>

#include "common.cuh"

namespace s1 {
namespace lin {

__device__ __forceinline__ float ld_f(const f16* p) { return __half2float(*p); }
__device__ __forceinline__ float ld_f(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_f(f16* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void st_f(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// exp of a head's log decay: at most 1, exactly 0 for -inf
__device__ __forceinline__ float decay(float log_decay) { return expf(fminf(log_decay, 0.f)); }

// Token by token, one warp per (sequence, head, value row): the state row in registers.
template <typename T, int DK, int N>
__global__ void __launch_bounds__(128)
    token_kernel(const __grid_constant__ SeqTab<N> tab, const LinAttnArgs a, int seq0) {
  constexpr int E = DK / 32;
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = w / a.dv, r = w % a.dv, s = blockIdx.y;
  const int64_t at = ((int64_t)h * a.dv + r) * DK + lane * E, per = (int64_t)a.H * a.dv * DK;
  float S[E];
#pragma unroll
  for (int e = 0; e < E; ++e) S[e] = a.S_in ? a.S_in[(int64_t)(seq0 + s) * a.s_in_stride + at + e] : 0.f;
  const float lam = decay(a.log_decay[h]);
  const int64_t row0 = tab.row0[s], n = tab.cum[s + 1] - tab.cum[s];
  for (int64_t t = row0; t < row0 + n; ++t) {
    const T* q = (const T*)a.q + t * a.q_stride + h * DK + lane * E;
    const T* k = (const T*)a.k + t * a.k_stride + h * DK + lane * E;
    const float v = ld_f((const T*)a.v + t * a.v_stride + h * a.dv + r);
    float o = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      S[e] = lam * S[e] + v * ld_f(k + e);
      o += S[e] * ld_f(q + e);
    }
    o = warp_sum(o);
    if (lane == 0) st_f((T*)a.out + (t * a.H + h) * a.dv + r, o * a.scale);
  }
  if (a.S_out) {
#pragma unroll
    for (int e = 0; e < E; ++e) a.S_out[(seq0 + s) * per + at + e] = S[e];
  }
}

// One token per sequence. A block takes 32 value rows of one (sequence, head), a warp 8 of them:
// the state is read and written once, coalesced rows of dk floats.
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

int64_t linattn_ws_bytes(int, const int*, int, int, int, int) { return 0; }

template <int N>
static cudaError_t lin_group(const LinAttnArgs& a, const SeqTab<N>& tab, int seq0, cudaStream_t st) {
  const dim3 grid(a.H * a.dv / 4, tab.n), block(128);
  if (a.dtype == ELEM_F16)
    return a.dk == 128 ? launch_pdl(lin::token_kernel<f16, 128, N>, grid, block, 0, st, tab, a, seq0)
                       : launch_pdl(lin::token_kernel<f16, 64, N>, grid, block, 0, st, tab, a, seq0);
  return a.dk == 128 ? launch_pdl(lin::token_kernel<bf16, 128, N>, grid, block, 0, st, tab, a, seq0)
                     : launch_pdl(lin::token_kernel<bf16, 64, N>, grid, block, 0, st, tab, a, seq0);
}

cudaError_t launch_linattn(const LinAttnArgs& a, int n_seq, const int* row0, const int* len, int, cudaStream_t st) {
  int s = 0;
  while (s < n_seq) {
    const int seq0 = s;
    SeqTab<SEQ_TAB_LARGE> t;
    t.n = 0;
    t.cum[0] = 0;
    for (; s < n_seq && t.n < SEQ_TAB_LARGE; ++s) {
      if ((int64_t)t.cum[t.n] + len[s] > INT32_MAX) break;
      t.row0[t.n] = row0[s];
      t.cum[t.n + 1] = t.cum[t.n] + len[s];
      ++t.n;
    }
    if (t.n <= SEQ_TAB_SMALL) {
      SeqTab<SEQ_TAB_SMALL> u;
      u.n = t.n;
      std::copy(t.cum, t.cum + t.n + 1, u.cum);
      std::copy(t.row0, t.row0 + t.n, u.row0);
      CK_RET(lin_group(a, u, seq0, st));
    } else {
      CK_RET(lin_group(a, t, seq0, st));
    }
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
