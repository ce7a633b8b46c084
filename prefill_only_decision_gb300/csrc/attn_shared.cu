// Attention of a batch of sequences over one shared prefix.
//
// Query row i of sequence s attends to the P rows of the snapshot and to rows 0 .. i of its own
// sequence: o = softmax(scale q.k) v with a running maximum and sum in fp32.
#include <algorithm>
#include <vector>

#include <cuda_fp8.h>

#include "common.cuh"

namespace s1 {
namespace sha {

// One warp per (query row, q head); each lane holds hd / 32 elements of q and of the output.
template <int HD, bool E4M3, int N>
__global__ void __launch_bounds__(128)
    simple_kernel(const __grid_constant__ SeqTab<N> tab, const SharedAttnArgs a) {
  constexpr int E = HD / 32;
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int vr = (int)(w / a.Hq), h = (int)(w % a.Hq), g = h / (a.Hq / a.Hkv);
  if (vr >= tab.cum[tab.n]) return;
  int s = 0;
  while (tab.cum[s + 1] <= vr) ++s;
  const int64_t first = tab.row0[s], row = first + vr - tab.cum[s];
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = h2f(a.q[row * a.q_stride + h * HD + lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  auto key = [&](const float* k, const float* v) {
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += q[e] * k[e];
    z = warp_sum(z);
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - base), p = expf(z - base);
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * v[e];
    m = mn;
  };
  float k[E], v[E];
  for (int j = 0; j < a.P; ++j) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t ki = ((int64_t)j * a.Hkv + g) * HD + lane * E + e;
      const int64_t vi = (((int64_t)a.cap + j) * a.Hkv + g) * HD + lane * E + e;
      if constexpr (E4M3) {
        const uint8_t* c = (const uint8_t*)a.kv;
        auto val = [&](int64_t at, float sc) {
          const float x = __half2float(__half(__nv_cvt_fp8_to_halfraw(c[at], __NV_E4M3))) * sc;
          return h2f(f2h(fabsf(x) > 65504.f ? copysignf(65504.f, x) : x));
        };
        k[e] = val(ki, a.scales[(int64_t)g * a.cap + j]);
        v[e] = val(vi, a.scales[((int64_t)a.Hkv + g) * a.cap + j]);
      } else {
        k[e] = h2f(((const f16*)a.kv)[ki]);
        v[e] = h2f(((const f16*)a.kv)[vi]);
      }
    }
    key(k, v);
  }
  if (a.kn)
    for (int64_t j = first; j <= row; ++j) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = h2f(a.kn[j * a.kv_stride + g * HD + lane * E + e]);
        v[e] = h2f(a.vn[j * a.kv_stride + g * HD + lane * E + e]);
      }
      key(k, v);
    }
  const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[(row * a.Hq + h) * HD + lane * E + e] = f2h(o[e] * inv);
}

}  // namespace sha

int64_t attention_shared_ws_bytes(int, const int*, int, int, int, int, int) { return 0; }

template <int N>
static cudaError_t shared_group(const SharedAttnArgs& a, const SeqTab<N>& tab, cudaStream_t st) {
  const int64_t warps = (int64_t)tab.cum[tab.n] * a.Hq;
  const dim3 grid((unsigned)((warps + 3) / 4)), block(128);
  if (a.hd == 128)
    return a.e4m3 ? launch_pdl(sha::simple_kernel<128, true, N>, grid, block, 0, st, tab, a)
                  : launch_pdl(sha::simple_kernel<128, false, N>, grid, block, 0, st, tab, a);
  return a.e4m3 ? launch_pdl(sha::simple_kernel<64, true, N>, grid, block, 0, st, tab, a)
                : launch_pdl(sha::simple_kernel<64, false, N>, grid, block, 0, st, tab, a);
}

cudaError_t launch_attention_shared(const SharedAttnArgs& a, int n_seq, const int* row0, const int* len, int,
                                    cudaStream_t st) {
  int s = 0;
  while (s < n_seq) {
    SeqTab<SEQ_TAB_LARGE> t;
    t.n = 0;
    t.cum[0] = 0;
    for (; s < n_seq && t.n < SEQ_TAB_LARGE; ++s) {
      if (len[s] == 0) continue;
      if ((int64_t)t.cum[t.n] + len[s] > INT32_MAX) break;
      t.row0[t.n] = row0[s];
      t.cum[t.n + 1] = t.cum[t.n] + len[s];
      ++t.n;
    }
    if (t.n == 0) continue;
    if (t.n <= SEQ_TAB_SMALL) {
      SeqTab<SEQ_TAB_SMALL> u;
      u.n = t.n;
      std::copy(t.cum, t.cum + t.n + 1, u.cum);
      std::copy(t.row0, t.row0 + t.n, u.row0);
      CK_RET(shared_group(a, u, st));
    } else {
      CK_RET(shared_group(a, t, st));
    }
  }
  return cudaSuccess;
}

}  // namespace s1
