// Argument checks shared by the C ABI files of the 8-bit and 4-bit operators and
// of the expert routing.
#pragma once

#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace dg {

constexpr int64_t kMaxSize = int64_t(1) << 30;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool type16(dg_dtype t) { return t == DG_F16 || t == DG_BF16; }

inline dg_status bad(const char* msg) { return set_error(DG_ERR_INVALID_ARG, msg); }

inline dg_status check_sizes(int64_t a, int64_t b, int64_t c) {
  if (a < 0 || b < 0 || c < 0) return bad("negative size");
  if (a > kMaxSize || b > kMaxSize || c > kMaxSize) return bad("size above 2^30");
  return DG_OK;
}

// 16-bit rows: 16-byte aligned base, pitch >= width and a multiple of 8.
inline dg_status check_rows16(const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p) return set_errorf(DG_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned16(p)) return set_errorf(DG_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (ld < width || ld % 8 != 0)
    return set_errorf(DG_ERR_INVALID_ARG,
                      "%s: row pitch %lld must be >= %lld elements and a multiple of 8", name,
                      (long long)ld, (long long)width);
  return DG_OK;
}

// D, the scalars and the epilogue of a product with N columns; *flags gets
// the kernels' epilogue flags.
inline dg_status check_output(const void* D, dg_dtype dtype, int64_t ldd, int64_t N, const void* bias,
                       float alpha, float beta, dg_epilogue epilogue, int* flags) {
  if (epilogue < DG_EPI_NONE || epilogue > DG_EPI_BIAS_GELU)
    return set_errorf(DG_ERR_INVALID_ARG, "unknown epilogue %d", static_cast<int>(epilogue));
  *flags = ((epilogue == DG_EPI_BIAS || epilogue == DG_EPI_BIAS_GELU) ? kEpiBias : 0) |
           ((epilogue == DG_EPI_GELU || epilogue == DG_EPI_BIAS_GELU) ? kEpiGelu : 0);
  if (!type16(dtype) && dtype != DG_F32)
    return set_errorf(DG_ERR_UNSUPPORTED, "D is F16, BF16 or F32, not %d", static_cast<int>(dtype));
  if (!D) return bad("D is null");
  if (!aligned16(D)) return bad("D is not 16-byte aligned");
  if (ldd < N)
    return set_errorf(DG_ERR_INVALID_ARG, "ldd (%lld) < N (%lld)", (long long)ldd, (long long)N);
  if (!(isfinite(alpha) && isfinite(beta))) return bad("alpha and beta must be finite");
  if (*flags & kEpiBias) {
    if (!bias) return bad("bias epilogue with a null bias");
    if (reinterpret_cast<uintptr_t>(bias) & (dtype == DG_F32 ? 3u : 1u))
      return bad("bias is not aligned to its type");
  }
  return DG_OK;
}

// Rows x top_k slots of a routing, and the count of experts where one is given.
inline dg_status check_routing(int64_t tokens, int64_t top_k, int64_t rows) {
  if (tokens < 0 || top_k < 1 || rows < 0) return bad("tokens and rows must be >= 0, top_k >= 1");
  if (top_k > 1024 || tokens > kMaxSize / top_k || rows > kMaxSize)
    return bad("top_k above 1024, or more than 2^30 slots or rows");
  return DG_OK;
}

inline dg_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DG_OK;
  if (e == cudaErrorInvalidConfiguration) {
    cudaGetLastError();
    return set_errorf(DG_ERR_UNSUPPORTED, "%s: more than 2^30 tiles or CTAs", what);
  }
  return set_cuda_error(e, what);
}

}  // namespace dg
