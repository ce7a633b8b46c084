// Stream-ordered operators over a long shared prefix (s1_ops.h): argument checks and dispatch.
#include <new>

#include "giveups.h"
#include "ops_check.h"

using namespace s1::opc;
using namespace s1;

namespace {
// The kernels' words side by side, for one copy to the host (a copy each: 36 us a call of s1_op_sync on an idle stream
// with four of them, 19 with two).
struct Words {
  uint64_t* at[4];
};
__device__ uint64_t g_now[4];
__global__ void gather_words(const Words w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (threadIdx.x == i) g_now[i] = *(volatile uint64_t*)w.at[i];
}

// Checks shared by both directions of the 8-bit snapshot. *skip: nothing to do.
int check_kv(const void* k, const void* v, int32_t dtype, int64_t ks, int64_t vs, int32_t n_rows,
             int32_t Hkv, int32_t hd, const void* codes, const void* scales, int32_t cap, int32_t pos0, bool* skip) {
  *skip = false;
  if (dtype != S1_F16 && dtype != S1_BF16 && dtype != S1_F32) return bad("kv: dtype must be S1_F16, S1_BF16 or S1_F32");
  if (n_rows < 0 || Hkv < 1 || cap < 0 || pos0 < 0 || (int64_t)pos0 + n_rows > cap)
    return bad("kv: rows outside the snapshot, or Hkv < 1");
  if (hd != 64 && hd != 128) return unsupported("kv: head dim must be 64 or 128");
  if (Hkv > 65536) return unsupported("kv: more than 65536 heads");
  if (ks < (int64_t)Hkv * hd || vs < (int64_t)Hkv * hd) return bad("kv: a row stride is below Hkv * hd");
  if (n_rows == 0) { *skip = true; return S1_OK; }
  if (!k || !v || !codes || !scales) return bad("kv: a NULL pointer");
  const size_t es = dtype == S1_F32 ? 4 : 2;
  if (!aligned(k, es) || !aligned(v, es) || !aligned(scales, 4) || !aligned(codes, 16))
    return bad("kv: misaligned pointer (codes 16 bytes, others their element)");
  return S1_OK;
}

int check_lin(const void* q, const void* k, const void* v, int32_t dtype, int64_t qs, int64_t ks, int64_t vs,
              const void* log_decay, int32_t n, int32_t H, int32_t dk, int32_t dv, const float* S_in,
              int64_t s_in_stride, const float* S_out, const void* out) {
  if (dtype != S1_F16 && dtype != S1_BF16) return bad("linattn: dtype must be S1_F16 or S1_BF16");
  if (n < 0 || H < 1) return bad("linattn: a negative sequence count, or H < 1");
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return unsupported("linattn: dk and dv must be 64 or 128");
  if (H > 4096) return unsupported("linattn: more than 4096 heads");
  const int64_t per = (int64_t)H * dk * dv;
  if (qs < (int64_t)H * dk || ks < (int64_t)H * dk || vs < (int64_t)H * dv)
    return bad("linattn: a row stride is below its heads' width");
  if ((qs | ks | vs) % 8) return bad("linattn: row strides must be multiples of 8 elements");
  if (S_in && s_in_stride != 0 && s_in_stride != per) return bad("linattn: s_in_stride must be 0 or H * dv * dk");
  if (n == 0) return S1_OK;
  if (!q || !k || !v || !log_decay || !out) return bad("linattn: a NULL pointer");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(S_in, 16) ||
      !aligned(S_out, 16) || !aligned(log_decay, 4))
    return bad("linattn: misaligned pointer (16 bytes; log_decay 4)");
  if (S_in && S_out) {
    const uintptr_t i0 = (uintptr_t)S_in, i1 = i0 + (size_t)(s_in_stride ? n : 1) * per * 4;
    const uintptr_t o0 = (uintptr_t)S_out, o1 = o0 + (size_t)n * per * 4;
    const bool in_place = i0 == o0 && (s_in_stride == per || n == 1);
    if (i0 < o1 && o0 < i1 && !in_place) return bad("linattn: S_out overlaps S_in (only in place, one state per sequence)");
  }
  return S1_OK;
}
}  // namespace

extern "C" {

int s1_op_sync(void* stream) {
  static GiveUps<4> told;
  cudaStream_t st = (cudaStream_t)stream;
  Words words = {};
  void* now_at = nullptr;
  int dev = 0;
  bool any = false;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = attention_shared_gave_up_word(&words.at[0]);
  if (e == cudaSuccess) e = linattn_gave_up_word(&words.at[1]);
  if (e == cudaSuccess) e = attention_step_gave_up_word(&words.at[2]);
  if (e == cudaSuccess) e = attention_paged_gave_up_word(&words.at[3]);
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&now_at, g_now);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess)
    e = (cudaError_t)told.news(dev, [&](uint64_t* now) {     // (one caller at a time: g_now is its own)
      gather_words<<<1, 4, 0, st>>>(words);
      cudaError_t r = cudaGetLastError();
      if (r == cudaSuccess) {
        r = cudaMemcpyAsync(now, now_at, sizeof(g_now), cudaMemcpyDeviceToHost, st);
      } else if (r == cudaErrorInvalidResourceHandle) {      // a stream of another device takes copies, but no kernel of this one
        r = cudaSuccess;
        for (int i = 0; i < 4 && r == cudaSuccess; ++i)
          r = cudaMemcpyAsync(&now[i], words.at[i], sizeof(now[i]), cudaMemcpyDeviceToHost, st);
      }
      if (r == cudaSuccess) r = cudaStreamSynchronize(st);
      return (int)r;
    }, &any);
  if (e != cudaSuccess) return cuda_rc(e, "op_sync");
  if (any) return s1::set_error(S1_ERR_DEVICE_TIMEOUT, "op_sync: a bounded device wait gave up");
  return S1_OK;
}

int s1_op_kv_quant_async(const void* k, const void* v, int32_t dtype, int64_t k_stride, int64_t v_stride,
                         int32_t n_rows, int32_t Hkv, int32_t hd, void* codes, float* scales, int32_t cap,
                         int32_t pos0, void* stream) {
  bool skip;
  const int rc = check_kv(k, v, dtype, k_stride, v_stride, n_rows, Hkv, hd, codes, scales, cap, pos0, &skip);
  if (rc != S1_OK || skip) return rc;
  return cuda_rc(launch_kv_quant(k, v, dtype, k_stride, v_stride, n_rows, Hkv, hd, (uint8_t*)codes, scales, cap, pos0,
                                 (cudaStream_t)stream),
                 "kv_quant");
}

int s1_op_kv_dequant_async(const void* codes, const float* scales, int32_t cap, int32_t pos0, int32_t n_rows,
                           int32_t Hkv, int32_t hd, void* k, void* v, int32_t dtype, int64_t k_stride,
                           int64_t v_stride, void* stream) {
  bool skip;
  const int rc =
      check_kv(k, v, dtype, k_stride, v_stride, n_rows, Hkv, hd, codes, scales, cap, pos0, &skip);
  if (rc != S1_OK || skip) return rc;
  return cuda_rc(launch_kv_dequant((const uint8_t*)codes, scales, cap, pos0, n_rows, Hkv, hd, k, v, dtype, k_stride,
                                   v_stride, (cudaStream_t)stream),
                 "kv_dequant");
}

static int check_shared_shape(int32_t n_seq, const int32_t* len, int32_t P, int32_t Hq, int32_t Hkv, int32_t hd) {
  if (n_seq < 0 || (n_seq > 0 && !len) || P < 0 || Hq < 1 || Hkv < 1)
    return bad("attention_shared: a negative count, a NULL array, or no heads");
  if (Hq % Hkv) return bad("attention_shared: Hq must be a multiple of Hkv");
  if (hd != 64 && hd != 128) return unsupported("attention_shared: head dim must be 64 or 128");
  if (Hq / Hkv > 128) return unsupported("attention_shared: more than 128 q heads per kv head");
  if (Hq > 32768) return unsupported("attention_shared: more than 32768 q heads");
  return S1_OK;
}

int s1_op_attention_shared_workspace(int32_t n_seq, const int32_t* len, int32_t P, int32_t Hq, int32_t Hkv,
                                     int32_t hd, int64_t* bytes) {
  if (!bytes) return bad("attention_shared_workspace: bytes is NULL");
  const int rc = check_shared_shape(n_seq, len, P, Hq, Hkv, hd);
  if (rc != S1_OK) return rc;
  if (const char* m = check_seqs(n_seq, nullptr, len)) return bad(m);
  *bytes = attention_shared_ws_bytes(n_seq, len, P, Hq, Hkv, hd, sm_count());
  return S1_OK;
}

int s1_op_attention_shared_async(const void* q, int64_t q_stride, const void* k_new, const void* v_new,
                                 int64_t kv_stride, int32_t n_seq, const int32_t* row0, const int32_t* len,
                                 const void* kv, const float* scales, int32_t kv_format, int32_t P, int32_t cap,
                                 int32_t Hq, int32_t Hkv, int32_t hd, float sm_scale, void* out, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  const int rc = check_shared_shape(n_seq, len, P, Hq, Hkv, hd);
  if (rc != S1_OK) return rc;
  if (kv_format != S1_KV_F16 && kv_format != S1_KV_E4M3) return bad("attention_shared: unknown kv_format");
  if (n_seq > 0 && !row0) return bad("attention_shared: row0 is NULL");
  if (const char* m = check_seqs(n_seq, row0, len)) return bad(m);
  if (P > cap) return bad("attention_shared: P is above the snapshot's capacity");
  if ((k_new == nullptr) != (v_new == nullptr)) return bad("attention_shared: k_new and v_new must both be given or both NULL");
  if (q_stride < (int64_t)Hq * hd || (k_new && kv_stride < (int64_t)Hkv * hd))
    return bad("attention_shared: a row stride is below its heads' width");
  if (q_stride % 8 || (k_new && kv_stride % 8)) return bad("attention_shared: row strides must be multiples of 8 elements");
  if (!(sm_scale > 0.f) || sm_scale > 3.4e38f) return bad("attention_shared: sm_scale must be positive and finite");
  int64_t rows = 0;
  for (int s = 0; s < n_seq; ++s) rows += len[s];
  if (rows == 0) return S1_OK;
  if (!q || !out) return bad("attention_shared: a NULL pointer");
  if (P > 0 && (!kv || (kv_format == S1_KV_E4M3 && !scales))) return bad("attention_shared: the snapshot is NULL");
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(kv, 16) || !aligned(out, 16) ||
      !aligned(scales, 4) || !aligned(workspace, 16))
    return bad("attention_shared: misaligned pointer (16 bytes; scales 4)");
  const int sms = sm_count();
  const int64_t need = attention_shared_ws_bytes(n_seq, len, P, Hq, Hkv, hd, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return bad("attention_shared: the workspace is too small");
  const SharedAttnArgs a{(const f16*)q, (const f16*)k_new, (const f16*)v_new, q_stride, kv_stride, kv, scales,
                         kv_format == S1_KV_E4M3, P, cap, Hq, Hkv, hd, sm_scale, (f16*)out, workspace};
  try {
    return cuda_rc(launch_attention_shared(a, n_seq, row0, len, sms, (cudaStream_t)stream), "attention_shared");
  } catch (const std::bad_alloc&) {
    return s1::set_error(S1_ERR_OOM, "attention_shared: host memory");
  }
}

int s1_op_linattn_workspace(int32_t n_seq, const int32_t* len, int32_t H, int32_t dk, int32_t dv, int64_t* bytes) {
  if (!bytes || n_seq < 0 || (n_seq > 0 && !len) || H < 1)
    return bad("linattn_workspace: a negative count, a NULL pointer, or H < 1");
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return unsupported("linattn: dk and dv must be 64 or 128");
  if (H > 4096) return unsupported("linattn: more than 4096 heads");
  if (const char* m = check_seqs(n_seq, nullptr, len)) return bad(m);
  *bytes = linattn_ws_bytes(n_seq, len, H, dk, dv, sm_count());
  return S1_OK;
}

int s1_op_linattn_async(const void* q, const void* k, const void* v, int32_t dtype, int64_t q_stride,
                        int64_t k_stride, int64_t v_stride, const float* log_decay, int32_t n_seq,
                        const int32_t* row0, const int32_t* len, int32_t H, int32_t dk, int32_t dv, float scale,
                        const float* S_in, int64_t s_in_stride, float* S_out, void* out, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  const int rc = check_lin(q, k, v, dtype, q_stride, k_stride, v_stride, log_decay, n_seq, H, dk, dv, S_in, s_in_stride,
                           S_out, out);
  if (rc != S1_OK || n_seq == 0) return rc;
  if (!row0 || !len) return bad("linattn: row0 or len is NULL");
  if (const char* m = check_seqs(n_seq, row0, len)) return bad(m);
  if (!aligned(workspace, 16)) return bad("linattn: misaligned workspace (16 bytes)");
  const int sms = sm_count();
  const int64_t need = linattn_ws_bytes(n_seq, len, H, dk, dv, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return bad("linattn: the workspace is too small");
  const LinAttnArgs a{q, k, v, dtype, q_stride, k_stride, v_stride, log_decay, H, dk, dv, scale,
                      S_in, s_in_stride, S_out, out, workspace};
  try {
    return cuda_rc(launch_linattn(a, n_seq, row0, len, sms, (cudaStream_t)stream), "linattn");
  } catch (const std::bad_alloc&) {
    return s1::set_error(S1_ERR_OOM, "linattn: host memory");
  }
}

int s1_op_linattn_step_async(const void* q, const void* k, const void* v, int32_t dtype, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const float* log_decay, int32_t n, int32_t H,
                             int32_t dk, int32_t dv, float scale, const float* S_in, int64_t s_in_stride,
                             float* S_out, void* out, void* stream) {
  const int rc =
      check_lin(q, k, v, dtype, q_stride, k_stride, v_stride, log_decay, n, H, dk, dv, S_in, s_in_stride, S_out, out);
  if (rc != S1_OK || n == 0) return rc;
  if ((int64_t)n * H * (dv / 32) > INT32_MAX) return unsupported("linattn_step: n * H * dv is above 32 * (2^31 - 1)");
  const LinAttnArgs a{q, k, v, dtype, q_stride, k_stride, v_stride, log_decay, H, dk, dv, scale,
                      S_in, s_in_stride, S_out, out, nullptr};
  return cuda_rc(launch_linattn_step(a, n, (cudaStream_t)stream), "linattn_step");
}

}  // extern "C"
