// Argument checks and errors that the stream-ordered operators' entry points share.
#pragma once
#include <cstdio>

#include "common.cuh"
#include "../../include/s1.h"
#include "../../include/s1_ops.h"

namespace s1 {
int set_error(int code, const char* msg);   // s1_api.cu: the thread-local message of s1_last_error

static_assert((int)ELEM_F32 == (int)S1_F32 && (int)ELEM_BF16 == (int)S1_BF16 && (int)ELEM_F16 == (int)S1_F16,
              "element types are the ABI's");

namespace opc {
inline int bad(const char* msg) { return set_error(S1_ERR_INVALID_ARG, msg); }
inline int unsupported(const char* msg) { return set_error(S1_ERR_UNSUPPORTED, msg); }
inline int cuda_rc(cudaError_t e, const char* op) {
  if (e == cudaSuccess) return S1_OK;
  cudaGetLastError();
  char b[256];
  snprintf(b, sizeof(b), "%s: %s", op, cudaGetErrorString(e));
  return set_error(S1_ERR_CUDA, b);
}
inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// SMs of the current device; without a device (host-side sizing) a GB300's.
inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    sms = 152;
  }
  return sms;
}

// Packed sequences: non-negative, ascending, disjoint, ends within 31 bits. NULL message: fine.
inline const char* check_seqs(int n_seq, const int32_t* row0, const int32_t* len) {
  int64_t end = 0;
  for (int s = 0; s < n_seq; ++s) {
    if (len[s] < 0) return "a sequence length is negative";
    if (!row0 || len[s] == 0) continue;
    if (row0[s] < end) return "sequences overlap, descend or start below row 0";
    end = (int64_t)row0[s] + len[s];
    if (end > INT32_MAX) return "a sequence ends past row 2^31 - 1";
  }
  return nullptr;
}
}  // namespace opc
}  // namespace s1
