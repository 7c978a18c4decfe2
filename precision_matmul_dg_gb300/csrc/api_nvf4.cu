// C ABI of the 4-bit operators with E4M3 block scales: argument checks and
// dispatch.
#include <math.h>

#include <algorithm>

#include "checks.h"
#include "dg.h"
#include "internal.h"

namespace dg {
namespace {

// Packed rows of `width` codes in matrices of `rows`, with their scales.
dg_status check_nvf4(const char* name, const void* codes, int64_t ld, int64_t width,
                     const void* scales, const float* row_scales) {
  if (!codes || !scales || !row_scales)
    return set_errorf(DG_ERR_INVALID_ARG, "%s or its scales is null", name);
  if (!aligned16(codes) || !aligned16(scales))
    return set_errorf(DG_ERR_INVALID_ARG, "%s or its scales is not 16-byte aligned", name);
  if (!aligned4(row_scales))
    return set_errorf(DG_ERR_INVALID_ARG, "%s: row scales are not 4-byte aligned", name);
  if (ld < ceil_div(width, 2) || ld % 16 != 0)
    return set_errorf(DG_ERR_INVALID_ARG,
                      "%s: row pitch %lld must be >= %lld bytes and a multiple of 16", name,
                      (long long)ld, (long long)ceil_div(width, 2));
  return DG_OK;
}

// The stride between the matrices of a stack, where there are several.
dg_status check_stack(const char* name, int64_t count, int64_t stride, int64_t rows, int64_t ld,
                      int64_t multiple) {
  if (count > 1 && (stride < rows * ld || stride % multiple != 0))
    return set_errorf(DG_ERR_INVALID_ARG,
                      "%s: the stride between matrices must be at least rows times the pitch and "
                      "a multiple of %lld",
                      name, (long long)multiple);
  return DG_OK;
}

// Sizes of a stack: every product that the kernels hold in 32 bits.
dg_status check_counts(int64_t count, int64_t rows, int64_t K) {
  dg_status s = check_sizes(count, rows, K);
  if (s != DG_OK) return s;
  if (count > 0 && ceil_div(rows, 128) * 128 > (int64_t(1) << 40) / count)
    return set_error(DG_ERR_UNSUPPORTED, "more than 2^40 rows in all");
  return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_quantize_nvf4(int64_t count, int64_t rows, int64_t K, dg_dtype dtype_x, const void* X,
                           int64_t ldx, int64_t stride_x, const float* given, void* codes,
                           int64_t ldq, int64_t stride_q, void* scales, float* row_scales,
                           dg_stream_t stream) {
  clear_error();
  dg_status s = check_counts(count, rows, K);
  if (s != DG_OK) return s;
  if (!type16(dtype_x))
    return set_errorf(DG_ERR_UNSUPPORTED, "X is F16 or BF16, not %d", static_cast<int>(dtype_x));
  if (count == 0 || rows == 0 || K == 0) return DG_OK;
  if ((s = check_rows16("X", X, ldx, K)) != DG_OK) return s;
  if ((s = check_stack("X", count, stride_x, rows, ldx, 8)) != DG_OK) return s;
  if ((s = check_nvf4("the codes", codes, ldq, K, scales, given ? given : row_scales)) != DG_OK)
    return s;
  if ((s = check_stack("the codes", count, stride_q, rows, ldq, 16)) != DG_OK) return s;
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  Nvf4RowsJob j;
  j.bf16 = dtype_x == DG_BF16;
  j.X = X;
  j.ldx = ldx;
  j.stride_x = count > 1 ? stride_x : 0;
  j.count = count;
  j.rows = rows;
  j.K = K;
  j.codes = codes;
  j.ldq = ldq;
  j.stride_q = count > 1 ? stride_q : 0;
  j.scales = scales;
  j.row_scales = row_scales;
  j.given = given;
  return launched(launch_quantize_nvf4(j, reinterpret_cast<cudaStream_t>(stream), c.sm_count),
                  "quantization launch");
}

dg_status dg_moe_dispatch_nvf4(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                               const void* X, int64_t ldx, int64_t rows, const int32_t* row_slot,
                               void* codes, int64_t ldq, void* scales, float* row_scales,
                               dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype)) return set_error(DG_ERR_UNSUPPORTED, "rows are F16 or BF16");
  if (rows == 0 || width == 0) return DG_OK;
  if (!row_slot || !aligned4(row_slot)) return bad("row_slot is null or not 4-byte aligned");
  if (tokens > 0 && (s = check_rows16("X", X, ldx, width)) != DG_OK) return s;
  if ((s = check_nvf4("the codes", codes, ldq, width, scales, row_scales)) != DG_OK) return s;
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  Nvf4RowsJob j;
  j.bf16 = dtype == DG_BF16;
  j.X = X;
  j.ldx = ldx;
  j.count = 1;
  j.rows = rows;
  j.K = width;
  j.codes = codes;
  j.ldq = ldq;
  j.scales = scales;
  j.row_scales = row_scales;
  j.row_slot = row_slot;
  j.top_k = top_k;
  j.tokens = tokens;
  return launched(launch_quantize_nvf4(j, reinterpret_cast<cudaStream_t>(stream), c.sm_count),
                  "dispatch launch");
}

dg_status dg_dequantize_nvf4(int64_t count, int64_t rows, int64_t K, const void* codes, int64_t ldq,
                             int64_t stride_q, const void* scales, const float* row_scales, void* D,
                             dg_dtype dtype_d, int64_t ldd, int64_t stride_d, dg_stream_t stream) {
  clear_error();
  dg_status s = check_counts(count, rows, K);
  if (s != DG_OK) return s;
  if (!type16(dtype_d) && dtype_d != DG_F32)
    return set_errorf(DG_ERR_UNSUPPORTED, "D is F16, BF16 or F32, not %d",
                      static_cast<int>(dtype_d));
  if (count == 0 || rows == 0 || K == 0) return DG_OK;
  if ((s = check_nvf4("the codes", codes, ldq, K, scales, row_scales)) != DG_OK) return s;
  if ((s = check_stack("the codes", count, stride_q, rows, ldq, 16)) != DG_OK) return s;
  if (!D || (reinterpret_cast<uintptr_t>(D) & (dtype_d == DG_F32 ? 3u : 1u)))
    return bad("D is null or not aligned to its type");
  if (ldd < K) return set_errorf(DG_ERR_INVALID_ARG, "ldd (%lld) < K (%lld)", (long long)ldd,
                                 (long long)K);
  if (count > 1 && stride_d < (rows - 1) * ldd + K)
    return bad("stride_d is too small: the matrices overlap");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  const Nvf4ValuesJob j = {count,  rows,       K, codes,   ldq, count > 1 ? stride_q : 0,
                           scales, row_scales, D, dtype_d, ldd, count > 1 ? stride_d : 0};
  return launched(launch_dequantize_nvf4(j, reinterpret_cast<cudaStream_t>(stream), c.sm_count),
                  "dequantization launch");
}

dg_status dg_gemm_nvf4(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                       const void* scale_a, const float* row_a, const void* B, int64_t ldb,
                       const void* scale_b, const float* row_b, void* D, dg_dtype dtype_d,
                       int64_t ldd, const void* bias, float alpha, float beta,
                       dg_epilogue epilogue, dg_stream_t stream) {
  clear_error();
  dg_status s = check_sizes(M, N, K);
  if (s != DG_OK) return s;
  if (M == 0 || N == 0) return DG_OK;
  if (K == 0) return bad("K must be at least 1");
  Nvf4Args a{};
  if ((s = check_output(D, dtype_d, ldd, N, bias, alpha, beta, epilogue, &a.epi)) != DG_OK)
    return s;
  if ((s = check_nvf4("A", A, lda, K, scale_a, row_a)) != DG_OK) return s;
  if ((s = check_nvf4("B", B, ldb, K, scale_b, row_b)) != DG_OK) return s;
  if (ceil_div(std::max(M, N), 128) * ceil_div(K, 64) > INT32_MAX)
    return set_error(DG_ERR_UNSUPPORTED, "more than 2^31 scale tiles");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.M = M;
  a.N = N;
  a.K = K;
  a.A = A;
  a.lda = lda;
  a.sa = scale_a;
  a.row_a = row_a;
  a.B = B;
  a.ldb = ldb;
  a.sb = scale_b;
  a.row_b = row_b;
  a.count = 1;
  a.D = D;
  a.dtype_d = dtype_d;
  a.ldd = ldd;
  a.bias = bias;
  a.alpha = alpha;
  a.beta = beta;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  a.status = c.status;
  a.timeout_ns = c.timeout_ns;
  a.sm_count = c.sm_count;
  return launched(launch_gemm_nvf4(a), "kernel launch");
}

dg_status dg_gemm_nvf4_grouped(int64_t count, int64_t rows, int64_t N, int64_t K, const void* A,
                               int64_t lda, const void* scale_a, const float* row_a, const void* B,
                               int64_t ldb, int64_t stride_b, const void* scale_b,
                               const float* row_b, const int32_t* offsets, void* D,
                               dg_dtype dtype_d, int64_t ldd, const void* bias,
                               int64_t stride_bias, float alpha, float beta, dg_epilogue epilogue,
                               dg_stream_t stream) {
  clear_error();
  dg_status s = check_sizes(rows, N, K);
  if (s != DG_OK) return s;
  if (count < 0) return bad("negative count");
  if (count > kMaxExperts)
    return set_errorf(DG_ERR_UNSUPPORTED, "more than %lld experts", (long long)kMaxExperts);
  if (count == 0 || rows == 0 || N == 0) return DG_OK;
  if (K == 0) return bad("K must be at least 1");
  Nvf4Args a{};
  if ((s = check_output(D, dtype_d, ldd, N, bias, alpha, beta, epilogue, &a.epi)) != DG_OK)
    return s;
  if (!offsets || !aligned4(offsets)) return bad("offsets is null or not 4-byte aligned");
  if ((s = check_nvf4("A", A, lda, K, scale_a, row_a)) != DG_OK) return s;
  if ((s = check_nvf4("B", B, ldb, K, scale_b, row_b)) != DG_OK) return s;
  if (count > 1 && (stride_b % ldb != 0 || stride_b / ldb < N))
    return bad("stride_b must be a multiple of ldb and at least N * ldb");
  if ((count > 1 ? (count - 1) * (stride_b / ldb) : 0) + N > INT32_MAX ||
      std::max(ceil_div(rows, 128), count * ceil_div(N, 128)) * ceil_div(K, 64) > INT32_MAX)
    return set_error(DG_ERR_UNSUPPORTED, "more than 2^31 rows of weights or scale tiles");
  if ((a.epi & kEpiBias) && stride_bias < 0) return bad("negative stride_bias");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.M = rows;
  a.N = N;
  a.K = K;
  a.A = A;
  a.lda = lda;
  a.sa = scale_a;
  a.row_a = row_a;
  a.B = B;
  a.ldb = ldb;
  a.stride_b = count > 1 ? stride_b : N * ldb;
  a.sb = scale_b;
  a.row_b = row_b;
  a.count = count;
  a.offsets = offsets;
  a.D = D;
  a.dtype_d = dtype_d;
  a.ldd = ldd;
  a.bias = bias;
  a.stride_bias = stride_bias;
  a.alpha = alpha;
  a.beta = beta;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  a.status = c.status;
  a.timeout_ns = c.timeout_ns;
  a.sm_count = c.sm_count;
  return launched(launch_gemm_nvf4(a), "kernel launch");
}

}  // extern "C"
