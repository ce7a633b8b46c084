// Attention over a paged K/V cache: prompts and single tokens, with a sliding window and sinks.
//
// The simplest right form: a warp per (query row, q head) takes the visible rows one by one with a running maximum and sum.
#include <algorithm>
#include <climits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kvrows.cuh"

namespace s1 {
namespace pga {

constexpr int TAB = 1024;
// Packed sequences of one launch by value: rows of sequence seq[i] are row0[i] .. row0[i] + cum[i + 1] - cum[i] - 1.
struct PromptTab {
  int n;
  int cum[TAB + 1];
  int row0[TAB], pos0[TAB], seq[TAB];
};

template <typename T>
__global__ void __launch_bounds__(256)
    simple_kernel(const __grid_constant__ PromptTab tab, const __grid_constant__ PagedAttnArgs a, const int* pos, int n) {
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t rows = pos ? n : tab.cum[tab.n];
  if (item >= rows * a.Hq) return;
  const int v = (int)(item / a.Hq), h = (int)(item % a.Hq);
  int s = v, p, row = v;
  if (pos) {
    p = pos[v];
  } else {
    int i = 0;
    while (tab.cum[i + 1] <= v) ++i;
    row = tab.row0[i] + v - tab.cum[i];
    p = tab.pos0[i] + v - tab.cum[i];
    s = tab.seq[i];
  }
  const PagesArgs& pg = a.pages;
  const int kvh = h / (a.Hq / pg.Hkv), E = pg.hd / 32;
  float q[4], o[4] = {};
  for (int e = 0; e < E; ++e)
    q[e] = kvc::to_f(((const T*)a.q)[row * a.q_stride + (int64_t)h * pg.hd + e * 32 + lane]);
  float m = -INFINITY, l = 0.f;
  const int64_t end = min((int64_t)p + 1, (int64_t)pg.cols << pg.shift);
  for (int64_t j = 0; j < end; ++j) {
    if (a.window && p - j >= a.window && j >= a.sinks) {
      j = p - a.window;                      // (the next is the window's first)
      continue;
    }
    const int id = pg.table[s * pg.table_stride + (j >> pg.shift)];
    const bool ok = id >= 0 && id < pg.n_pages;
    const int64_t vec = (((int64_t)id * pg.Hkv + kvh) << pg.shift) + (j & ((1 << pg.shift) - 1));
    const int64_t plane = ((int64_t)pg.n_pages * pg.Hkv) << pg.shift;
    float k[4], vv[4], dot = 0.f;
    for (int e = 0; e < E; ++e) {
      const int64_t i0 = vec * pg.hd + e * 32 + lane, i1 = i0 + plane * pg.hd;
      k[e] = vv[e] = 0.f;
      if (!ok) continue;
      if (pg.format == KVF_E4M3) {
        const auto dec = [&](int64_t i) {
          return __half2float(__half(__nv_cvt_fp8_to_halfraw(((const __nv_fp8_storage_t*)pg.data)[i], __NV_E4M3)));
        };
        k[e] = dec(i0) * pg.scales[vec];
        vv[e] = dec(i1) * pg.scales[vec + plane];
      } else if (pg.format == KVF_BF16) {
        k[e] = bf2f(((const bf16*)pg.data)[i0]);
        vv[e] = bf2f(((const bf16*)pg.data)[i1]);
      } else {
        k[e] = h2f(((const f16*)pg.data)[i0]);
        vv[e] = h2f(((const f16*)pg.data)[i1]);
      }
    }
    for (int e = 0; e < E; ++e) dot += q[e] * k[e];
    const float z = warp_sum(dot) * a.scale;
    const float M = fmaxf(m, z);
    if (M == -INFINITY) continue;
    const float alpha = m == M ? 1.f : expf(m - M), w = z == M ? 1.f : expf(z - M);
    l = l * alpha + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + w * vv[e];
    m = M;
  }
  for (int e = 0; e < E; ++e) {
    const float y = l == 0.f ? 0.f : o[e] / l;
    T* dst = (T*)a.out + ((int64_t)row * a.Hq + h) * pg.hd + e * 32 + lane;
    if constexpr (std::is_same<T, f16>::value) *dst = f2h(y);
    else *dst = f2bf(y);
  }
}

cudaError_t launch_simple(const PromptTab& t, const PagedAttnArgs& a, const int* pos, int n, cudaStream_t st) {
  const int64_t warps = (int64_t)(pos ? n : t.cum[t.n]) * a.Hq;
  if ((warps + 7) / 8 > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(a.bf16 ? simple_kernel<bf16> : simple_kernel<f16>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st,
                    t, a, pos, n);
}
}  // namespace pga

cudaError_t launch_attention_paged(const PagedAttnArgs& a, int n_seq, const int* row0, const int* len, const int* pos0,
                                   int, cudaStream_t st) {
  pga::PromptTab t;
  for (int s = 0; s < n_seq;) {
    t.n = 0;
    t.cum[0] = 0;
    for (; s < n_seq && t.n < pga::TAB; ++s) {
      if (len[s] == 0) continue;
      t.row0[t.n] = row0[s];
      t.pos0[t.n] = pos0[s];
      t.seq[t.n] = s;
      t.cum[t.n + 1] = t.cum[t.n] + len[s];
      ++t.n;
    }
    if (t.n) CK_RET(pga::launch_simple(t, a, nullptr, 0, st));
  }
  return cudaSuccess;
}
int64_t attention_paged_ws_bytes(int, const int*, const int*, int, int, int, int, int, int) { return 0; }

}  // namespace s1
