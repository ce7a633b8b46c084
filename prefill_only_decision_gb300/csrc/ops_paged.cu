// Stream-ordered operators around a paged K/V cache (s1_ops.h): argument checks and dispatch.
#include <algorithm>
#include <cmath>
#include <new>

#include "ops_check.h"

using namespace s1::opc;
using namespace s1;

namespace {
bool elem(int32_t t) { return t == S1_F16 || t == S1_BF16 || t == S1_F32; }
size_t elem_bytes(int32_t t) { return t == S1_F32 ? 4 : 2; }

constexpr double TWO_64 = 18446744073709551616.0, FREQ_MAX = 1099511627776.0;   // 2^64, 2^40
constexpr float SCALE_MAX = 2.35e38f;   // times log2 e within fp32's range (scores of 0 would be NaN past it)

int check_rope(const s1_rope_spec* r, int32_t hd, RopeArgs* out) {
  out->n_pairs = 0;
  if (!r) return S1_OK;
  if (r->n_pairs < 8 || r->n_pairs % 8 || r->n_pairs > hd / 2)
    return bad("rope: n_pairs must be a multiple of 8 from 8 to hd / 2");
  if (r->n_axes < 1 || r->n_axes > 4) return bad("rope: n_axes must be 1 .. 4");
  if (!r->inv_freq) return bad("rope: inv_freq is NULL");
  out->n_pairs = r->n_pairs;
  for (int i = 0; i < r->n_pairs; ++i) {
    if (!std::isfinite(r->inv_freq[i])) return bad("rope: a frequency is not finite");
    if (std::fabs(r->inv_freq[i]) > FREQ_MAX) return unsupported("rope: a frequency above 2^40 radians per position");
    if (r->axis && r->axis[i] >= r->n_axes) return bad("rope: an axis is not below n_axes");
    // w / 2 pi as hi + lo, so that its fraction is right to 2^-64 and not to a double's 2^-53 (up to FREQ_MAX: lo holds no
    // more beside a larger hi)
    const double w = std::fabs(r->inv_freq[i]), hi = w * 0.15915494309189535;
    const double lo = std::fma(w, 0.15915494309189535, -hi) + w * -9.839338337591243e-18;
    const double frac = (hi - std::floor(hi)) * TWO_64, rest = lo * TWO_64;   // 0 .. 2^64
    const uint64_t turn = (frac >= TWO_64 ? 0 : (uint64_t)frac) + (uint64_t)(int64_t)std::llround(rest);
    out->turn[i] = r->inv_freq[i] < 0 ? 0 - turn : turn;
    out->axis[i] = r->axis ? r->axis[i] : 0;
  }
  return S1_OK;
}

int check_pages(const s1_kv_pages* p, PagesArgs* out) {
  if (!p) return bad("pages: NULL");
  if (p->format != S1_KV_F16 && p->format != S1_KV_BF16 && p->format != S1_KV_E4M3) return bad("pages: unknown format");
  if (p->page_rows != 16 && p->page_rows != 32 && p->page_rows != 64 && p->page_rows != 128)
    return unsupported("pages: page_rows must be 16, 32, 64 or 128");
  if (p->hd != 64 && p->hd != 128) return unsupported("pages: head dim must be 64 or 128");
  if (p->Hkv < 1 || p->n_pages < 1 || p->n_seq < 0 || p->cols < 0) return bad("pages: a count is out of range");
  if (p->Hkv > 4096) return unsupported("pages: more than 4096 kv heads");
  if (p->table_stride < p->cols) return bad("pages: table_stride is below cols");
  if ((int64_t)p->cols * p->page_rows > (1 << 30)) return unsupported("pages: a table row of more than 2^30 cached rows");
  if (!p->data || (!p->table && p->n_seq > 0 && p->cols > 0)) return bad("pages: a NULL pointer");
  if ((p->format == S1_KV_E4M3) != (p->scales != nullptr)) return bad("pages: scales go with S1_KV_E4M3, and only with it");
  if (!aligned(p->data, 16) || !aligned(p->scales, 16) || !aligned(p->table, 4))
    return bad("pages: misaligned pointer (data and scales 16 bytes, table 4)");
  int shift = 4;
  while ((1 << shift) < p->page_rows) ++shift;
  *out = PagesArgs{p->data, p->scales, p->format, p->n_pages, shift, p->Hkv, p->hd, p->table, p->n_seq, p->cols,
                   p->table_stride};
  return S1_OK;
}

int check_heads(int32_t Hq, int32_t Hkv) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv) return bad("attention_paged: Hq must be a positive multiple of Hkv");
  if (Hq / Hkv > 128) return unsupported("attention_paged: more than 128 q heads per kv head");
  if (Hq > 32768) return unsupported("attention_paged: more than 32768 q heads");
  return S1_OK;
}

// Checks that both forms of the attention share.
int check_attn(const void* q, int32_t q_dtype, int64_t q_stride, int32_t Hq, const s1_kv_pages* pages, int32_t window,
               int32_t sinks, float sm_scale, const void* out, const void* ws, PagesArgs* pg) {
  int rc = check_pages(pages, pg);
  if (rc != S1_OK || (rc = check_heads(Hq, pages->Hkv)) != S1_OK) return rc;
  if (q_dtype != S1_F16 && q_dtype != S1_BF16) return bad("attention_paged: q_dtype must be S1_F16 or S1_BF16");
  if (pg->format != S1_KV_E4M3 && (pg->format == S1_KV_F16) != (q_dtype == S1_F16))
    return bad("attention_paged: q must have the pages' type");
  if (q_stride < (int64_t)Hq * pg->hd) return bad("attention_paged: q_stride is below Hq * hd");
  if (q_stride % 8) return bad("attention_paged: q_stride must be a multiple of 8 elements");
  if (window < 0 || sinks < 0) return bad("attention_paged: window or sinks is negative");
  if (!(sm_scale > 0.f) || sm_scale > 3.4e38f) return bad("attention_paged: sm_scale must be positive and finite");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16))
    return bad("attention_paged: misaligned pointer (q, out and workspace 16 bytes)");
  return S1_OK;
}
}  // namespace

extern "C" {

int s1_op_rope_async(const void* x, int32_t dtype, int64_t x_stride, int32_t n_rows, int32_t H, int32_t hd,
                     const s1_rope_spec* rope, const int32_t* pos, int64_t pos_stride, void* out, int32_t out_dtype,
                     int64_t out_stride, void* stream) {
  if (!elem(dtype) || !elem(out_dtype)) return bad("rope: a dtype must be S1_F16, S1_BF16 or S1_F32");
  if (out_dtype != dtype && dtype != S1_F32) return bad("rope: 16-bit rows keep their type");
  if (n_rows < 0 || H < 1) return bad("rope: a negative row count, or H < 1");
  if (hd != 64 && hd != 128) return unsupported("rope: head dim must be 64 or 128");
  if (H > 65536) return unsupported("rope: more than 65536 heads");
  if (x_stride < (int64_t)H * hd || out_stride < (int64_t)H * hd) return bad("rope: a row stride is below H * hd");
  if (!rope) return bad("rope: the rotation is NULL");
  RowsArgs a = {};
  const int rc = check_rope(rope, hd, &a.rope);
  if (rc != S1_OK) return rc;
  if (rope->n_axes > 1 && pos_stride < n_rows) return bad("rope: pos_stride is below n_rows");
  if (n_rows == 0) return S1_OK;
  if (!x || !pos || !out) return bad("rope: a NULL pointer");
  if (!aligned(x, elem_bytes(dtype)) || !aligned(out, elem_bytes(out_dtype)) || !aligned(pos, 4))
    return bad("rope: misaligned pointer");
  if (out == x && (out_dtype != dtype || out_stride != x_stride)) return bad("rope: in place needs one type and one stride");
  a.q = x;
  a.q_stride = x_stride;
  a.n_rows = n_rows;
  a.Hq = H;
  a.hd = hd;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.q_out = out;
  a.q_out_type = out_dtype;
  a.q_out_stride = out_stride;
  return cuda_rc(launch_rope_rows(a, dtype, sm_count(), (cudaStream_t)stream), "rope");
}

int s1_op_kv_append_async(const void* q, const void* k, const void* v, int32_t dtype, int64_t q_stride, int64_t k_stride,
                          int64_t v_stride, int32_t n_rows, int32_t Hq, const s1_rope_spec* rope, const int32_t* pos,
                          int64_t pos_stride, const int32_t* seq, const int32_t* at, const s1_kv_pages* pages, void* q_out,
                          int32_t q_dtype, void* stream) {
  RowsArgs a = {};
  int rc = check_pages(pages, &a.pages);
  if (rc != S1_OK) return rc;
  const int64_t hd = pages->hd;
  if (!elem(dtype)) return bad("kv_append: dtype must be S1_F16, S1_BF16 or S1_F32");
  if (q_dtype != S1_F16 && q_dtype != S1_BF16) return bad("kv_append: q_dtype must be S1_F16 or S1_BF16");
  if (n_rows < 0 || Hq < 0) return bad("kv_append: a negative count");
  if (Hq > 32768) return unsupported("kv_append: more than 32768 q heads");
  if ((rc = check_rope(rope, pages->hd, &a.rope)) != S1_OK) return rc;
  if (Hq > 0 && q_stride < Hq * hd) return bad("kv_append: q_stride is below Hq * hd");
  if (k_stride < pages->Hkv * hd || v_stride < pages->Hkv * hd) return bad("kv_append: a row stride is below Hkv * hd");
  if (rope && pos && rope->n_axes > 1 && pos_stride < n_rows) return bad("kv_append: pos_stride is below n_rows");
  if (!seq && n_rows > pages->n_seq) return bad("kv_append: more rows than sequences, and seq is NULL");
  if ((Hq > 0) != (q != nullptr) && n_rows > 0) return bad("kv_append: q and Hq must both be given, or neither");
  if (n_rows == 0) return S1_OK;
  if (!k || !v || !at || (q && !q_out)) return bad("kv_append: a NULL pointer");
  const size_t es = elem_bytes(dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(q_out, 2) || !aligned(pos, 4) || !aligned(seq, 4) ||
      !aligned(at, 4))
    return bad("kv_append: misaligned pointer (its element)");
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q ? q_stride : 0;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_rows = n_rows;
  a.Hq = Hq;
  a.hd = pages->hd;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.seq = seq;
  a.at = at;
  a.q_out = q_out;
  a.q_out_type = q_dtype;
  a.q_out_stride = Hq * hd;
  return cuda_rc(launch_rope_rows(a, dtype, sm_count(), (cudaStream_t)stream), "kv_append");
}

int s1_op_attention_paged_step_workspace(int32_t n, int32_t Hq, int32_t Hkv, int32_t hd, int64_t* bytes) {
  if (!bytes || n < 0) return bad("attention_paged_step_workspace: bytes is NULL, or n is negative");
  const int rc = check_heads(Hq, Hkv);
  if (rc != S1_OK) return rc;
  if (hd != 64 && hd != 128) return unsupported("attention_paged: head dim must be 64 or 128");
  *bytes = attention_paged_step_ws_bytes(hd, sm_count());
  return S1_OK;
}

int s1_op_attention_paged_step_async(const void* q, int32_t q_dtype, int64_t q_stride, int32_t n, int32_t Hq,
                                     const s1_kv_pages* pages, const int32_t* pos, int32_t window, int32_t sinks,
                                     float sm_scale, void* out, void* workspace, int64_t workspace_bytes, void* stream) {
  PagedAttnArgs a = {};
  const int rc = check_attn(q, q_dtype, q_stride, Hq, pages, window, sinks, sm_scale, out, workspace, &a.pages);
  if (rc != S1_OK) return rc;
  if (n < 0 || n > pages->n_seq) return bad("attention_paged_step: n must be 0 .. n_seq");
  if ((int64_t)n * pages->Hkv * ((Hq / pages->Hkv + 15) / 16) * (((int64_t)pages->cols << a.pages.shift) / 64 + 2) > INT32_MAX)
    return unsupported("attention_paged_step: n * kv heads * rows of the table is above 2^37");
  if (n == 0) return S1_OK;
  if (!q || !out || !pos) return bad("attention_paged_step: a NULL pointer");
  if (!aligned(pos, 4)) return bad("attention_paged_step: misaligned pos");
  const int sms = sm_count();
  const int64_t need = attention_paged_step_ws_bytes(pages->hd, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return bad("attention_paged_step: the workspace is too small");
  a.q = q;
  a.bf16 = q_dtype == S1_BF16;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.window = window;
  a.sinks = sinks;
  a.scale = std::min(sm_scale, SCALE_MAX);
  a.out = out;
  a.ws = workspace;
  return cuda_rc(launch_attention_paged_step(a, n, pos, sms, (cudaStream_t)stream), "attention_paged_step");
}

int s1_op_attention_paged_workspace(int32_t n_seq, const int32_t* len, const int32_t* pos0, int32_t Hq, int32_t Hkv,
                                    int32_t hd, int32_t window, int32_t sinks, int64_t* bytes) {
  if (!bytes || n_seq < 0 || (n_seq > 0 && (!len || !pos0)) || window < 0 || sinks < 0)
    return bad("attention_paged_workspace: a negative count, or a NULL pointer");
  const int rc = check_heads(Hq, Hkv);
  if (rc != S1_OK) return rc;
  if (hd != 64 && hd != 128) return unsupported("attention_paged: head dim must be 64 or 128");
  if (const char* m = check_seqs(n_seq, nullptr, len)) return bad(m);
  for (int s = 0; s < n_seq; ++s)
    if (pos0[s] < 0 || (int64_t)pos0[s] + len[s] > INT32_MAX) return bad("attention_paged: a position is out of range");
  for (int s = 0; s < n_seq; ++s)
    if (!attention_paged_fits(len[s], pos0[s], Hq, Hkv))
      return unsupported("attention_paged: a sequence of too many rows x heads for one call");
  try {
    *bytes = attention_paged_ws_bytes(n_seq, len, pos0, Hq, Hkv, hd, window, sinks, sm_count());
  } catch (const std::bad_alloc&) {
    return s1::set_error(S1_ERR_OOM, "attention_paged_workspace: host memory");
  }
  return S1_OK;
}

int s1_op_attention_paged_async(const void* q, int32_t q_dtype, int64_t q_stride, int32_t n_seq, const int32_t* row0,
                                const int32_t* len, const int32_t* pos0, int32_t Hq, const s1_kv_pages* pages,
                                int32_t window, int32_t sinks, float sm_scale, void* out, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  PagedAttnArgs a = {};
  const int rc = check_attn(q, q_dtype, q_stride, Hq, pages, window, sinks, sm_scale, out, workspace, &a.pages);
  if (rc != S1_OK) return rc;
  if (n_seq < 0 || n_seq > pages->n_seq) return bad("attention_paged: n_seq must be 0 .. the table's");
  if (n_seq > 0 && (!row0 || !len || !pos0)) return bad("attention_paged: row0, len or pos0 is NULL");
  if (const char* m = check_seqs(n_seq, row0, len)) return bad(m);
  int64_t rows = 0;
  for (int s = 0; s < n_seq; ++s) {
    rows += len[s];
    if (pos0[s] < 0 || (int64_t)pos0[s] + len[s] > ((int64_t)pages->cols << a.pages.shift))
      return bad("attention_paged: a sequence ends past its table row, or starts below position 0");
  }
  for (int s = 0; s < n_seq; ++s)
    if (!attention_paged_fits(len[s], pos0[s], Hq, pages->Hkv))
      return unsupported("attention_paged: a sequence of too many rows x heads for one call");
  if (rows == 0) return S1_OK;
  if (!q || !out) return bad("attention_paged: a NULL pointer");
  a.q = q;
  a.bf16 = q_dtype == S1_BF16;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.window = window;
  a.sinks = sinks;
  a.scale = std::min(sm_scale, SCALE_MAX);
  a.out = out;
  a.ws = workspace;
  const int sms = sm_count();
  try {
    bool too_small;
    const cudaError_t e =
        launch_attention_paged(a, n_seq, row0, len, pos0, sms, workspace_bytes, &too_small, (cudaStream_t)stream);
    if (too_small) return bad("attention_paged: the workspace is too small");
    return cuda_rc(e, "attention_paged");
  } catch (const std::bad_alloc&) {
    return s1::set_error(S1_ERR_OOM, "attention_paged: host memory");
  }
}

}  // extern "C"
