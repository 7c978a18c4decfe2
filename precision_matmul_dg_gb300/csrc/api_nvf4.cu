// C ABI of the 4-bit operators with E4M3 block scales and of the expert layer
// for few tokens: argument checks and dispatch.
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

constexpr int64_t kFp8Block = 128;

// A product's weights: count matrices of n rows of k values.
dg_status check_moe_weights(const char* name, const dg_moe_weights* w, bool nvf4, int64_t count,
                            int64_t n, int64_t k) {
  if (!w) return set_errorf(DG_ERR_INVALID_ARG, "%s is null", name);
  if (nvf4) {
    const dg_status s = check_nvf4(name, w->codes, w->ld, k, w->scales, w->row_scales);
    if (s != DG_OK) return s;
  } else {
    if (!w->codes || !w->scales)
      return set_errorf(DG_ERR_INVALID_ARG, "%s or its scales is null", name);
    if (!aligned16(w->codes) || !aligned4(w->scales))
      return set_errorf(DG_ERR_INVALID_ARG, "%s or its scales is not aligned", name);
    if (w->ld < k || w->ld % 16 != 0)
      return set_errorf(DG_ERR_INVALID_ARG,
                        "%s: row pitch %lld must be >= %lld bytes and a multiple of 16", name,
                        (long long)w->ld, (long long)k);
    if (w->lds < ceil_div(k, kFp8Block))
      return set_errorf(DG_ERR_INVALID_ARG, "%s: %lld scales per row, need %lld", name,
                        (long long)w->lds, (long long)ceil_div(k, kFp8Block));
    if (count > 1 && w->stride_s < ceil_div(n, kFp8Block) * w->lds)
      return set_errorf(DG_ERR_INVALID_ARG, "%s: stride_s must be at least ceil(n / 128) * lds",
                        name);
  }
  if (count > 1 && (w->stride % w->ld != 0 || w->stride / w->ld < n))
    return set_errorf(DG_ERR_INVALID_ARG, "%s: stride must be a multiple of ld and at least n * ld",
                      name);
  if ((count > 1 ? (count - 1) * (w->stride / w->ld) : 0) + n > INT32_MAX ||
      count * ceil_div(n, 128) * ceil_div(k, 64) > INT32_MAX)
    return set_errorf(DG_ERR_UNSUPPORTED, "%s: more than 2^31 rows or scale tiles", name);
  if (w->bias && (reinterpret_cast<uintptr_t>(w->bias) & 1u))
    return set_errorf(DG_ERR_INVALID_ARG, "%s: bias is not aligned to its type", name);
  if (w->bias && w->stride_bias < 0)
    return set_errorf(DG_ERR_INVALID_ARG, "%s: negative stride_bias", name);
  return DG_OK;
}

MoeWeights moe_weights(const dg_moe_weights& w, int64_t count) {
  return {w.codes,        w.ld,        count > 1 ? w.stride : 0, w.scales,
          w.lds,          count > 1 ? w.stride_s : 0,            w.row_scales,
          w.bias,         w.stride_bias};
}

// Sizes of a layer call; the kernels' unit numbers are 32-bit.
dg_status check_layer(int64_t tokens, int64_t top_k, int64_t hidden, int64_t out) {
  dg_status s = check_routing(tokens, top_k, 0);
  if (s == DG_OK) s = check_sizes(hidden, out, 0);
  if (s != DG_OK) return s;
  if (tokens * top_k > kMaxLayerSlots)
    return set_errorf(DG_ERR_UNSUPPORTED, "more than %lld slots", (long long)kMaxLayerSlots);
  if (std::max(hidden, out) > (int64_t(1) << 24))
    return set_error(DG_ERR_UNSUPPORTED, "hidden or out above 2^24");
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

int64_t dg_moe_layer_scratch(int64_t tokens, int64_t top_k, int64_t hidden, int64_t out) {
  clear_error();
  if (check_layer(tokens, top_k, hidden, out) != DG_OK) return -1;
  MoeLayerArgs a{};
  a.tokens = tokens;
  a.top_k = top_k;
  a.hidden = hidden;
  a.out = out;
  return moe_layer_scratch(a);
}

dg_status dg_moe_layer(int64_t tokens, int64_t top_k, int64_t count, int64_t width, int64_t hidden,
                       int64_t out, dg_dtype dtype, const void* X, int64_t ldx, const int32_t* ids,
                       const float* weights, dg_moe_format format, const dg_moe_weights* up,
                       const dg_moe_weights* down, dg_moe_activation activation, void* D,
                       int64_t ldd, void* scratch, int64_t scratch_bytes, dg_stream_t stream) {
  clear_error();
  dg_status s = check_layer(tokens, top_k, hidden, out);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (count < 1) return bad("count must be >= 1");
  if (count > kMaxExperts)
    return set_errorf(DG_ERR_UNSUPPORTED, "more than %lld experts", (long long)kMaxExperts);
  if (!type16(dtype))
    return set_errorf(DG_ERR_UNSUPPORTED, "X and D are F16 or BF16, not %d",
                      static_cast<int>(dtype));
  if (format != DG_MOE_FP8 && format != DG_MOE_NVF4) return bad("unknown format");
  if (activation != DG_MOE_GELU && activation != DG_MOE_SWIGLU) return bad("unknown activation");
  if (tokens == 0 || out == 0) return DG_OK;
  if (width < 1 || hidden < 1) return bad("width and hidden must be at least 1");
  const bool gated = activation == DG_MOE_SWIGLU, nvf4 = format == DG_MOE_NVF4;
  if (gated && nvf4 && hidden % 128 != 0)
    return set_error(DG_ERR_UNSUPPORTED, "SwiGLU on NVF4 weights needs hidden a multiple of 128");
  if ((s = check_rows16("X", X, ldx, width)) != DG_OK) return s;
  if ((s = check_rows16("D", D, ldd, out)) != DG_OK) return s;
  if (!ids || !aligned4(ids)) return bad("ids is null or not 4-byte aligned");
  if (!aligned4(weights)) return bad("weights is not 4-byte aligned");
  if ((s = check_moe_weights("up", up, nvf4, count, hidden * (gated ? 2 : 1), width)) != DG_OK)
    return s;
  if ((s = check_moe_weights("down", down, nvf4, count, out, hidden)) != DG_OK) return s;
  MoeLayerArgs a{};
  a.nvf4 = nvf4;
  a.gated = gated;
  a.bf16 = dtype == DG_BF16;
  a.tokens = tokens;
  a.top_k = top_k;
  a.count = count;
  a.width = width;
  a.hidden = hidden;
  a.out = out;
  if (!moe_layer_fits(a))
    return set_error(DG_ERR_UNSUPPORTED, "tokens x width do not fit a CTA's shared memory: "
                                         "dg_moe_sort and the grouped products take them");
  const int64_t need = moe_layer_scratch(a);
  if (!scratch || !aligned16(scratch)) return bad("the scratch is null or not 16-byte aligned");
  if (scratch_bytes < need)
    return set_errorf(DG_ERR_INVALID_ARG, "%lld bytes of scratch, need %lld",
                      (long long)scratch_bytes, (long long)need);
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.X = X;
  a.ldx = ldx;
  a.ids = ids;
  a.weights = weights;
  a.up = moe_weights(*up, count);
  a.down = moe_weights(*down, count);
  a.D = D;
  a.ldd = ldd;
  a.scratch = scratch;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  a.status = c.status;
  a.timeout_ns = c.timeout_ns;
  a.sm_count = c.sm_count;
  return launched(launch_moe_layer(a), "layer launch");
}

}  // extern "C"
