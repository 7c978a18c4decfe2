// C ABI of the FP8 and expert-routing operators: argument checks and dispatch.
#include <math.h>

#include <algorithm>

#include "dg.h"
#include "internal.h"

namespace dg {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;
constexpr int64_t kFp8Block = 128;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool type16(dg_dtype t) { return t == DG_F16 || t == DG_BF16; }

dg_status bad(const char* msg) { return set_error(DG_ERR_INVALID_ARG, msg); }

dg_status check_sizes(int64_t a, int64_t b, int64_t c) {
  if (a < 0 || b < 0 || c < 0) return bad("negative size");
  if (a > kMaxSize || b > kMaxSize || c > kMaxSize) return bad("size above 2^30");
  return DG_OK;
}

// 16-bit rows: 16-byte aligned base, pitch >= width and a multiple of 8.
dg_status check_rows16(const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p) return set_errorf(DG_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned16(p)) return set_errorf(DG_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (ld < width || ld % 8 != 0)
    return set_errorf(DG_ERR_INVALID_ARG,
                      "%s: row pitch %lld must be >= %lld elements and a multiple of 8", name,
                      (long long)ld, (long long)width);
  return DG_OK;
}

// FP8 rows of `width` codes with `blocks` scales each.
dg_status check_fp8(const char* name, const void* codes, int64_t ld, int64_t width,
                    const float* scales, int64_t lds) {
  if (!codes || !scales)
    return set_errorf(DG_ERR_INVALID_ARG, "%s or its scales is null", name);
  if (!aligned16(codes))
    return set_errorf(DG_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (!aligned4(scales))
    return set_errorf(DG_ERR_INVALID_ARG, "%s: scales are not 4-byte aligned", name);
  if (ld < width || ld % 16 != 0)
    return set_errorf(DG_ERR_INVALID_ARG,
                      "%s: row pitch %lld must be >= %lld bytes and a multiple of 16", name,
                      (long long)ld, (long long)width);
  if (lds < ceil_div(width, kFp8Block))
    return set_errorf(DG_ERR_INVALID_ARG, "%s: %lld scales per row, need %lld", name,
                      (long long)lds, (long long)ceil_div(width, kFp8Block));
  return DG_OK;
}

// D, the scalars and the epilogue of a product with N columns; *flags gets
// the kernels' epilogue flags.
dg_status check_output(const void* D, dg_dtype dtype, int64_t ldd, int64_t N, const void* bias,
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
dg_status check_routing(int64_t tokens, int64_t top_k, int64_t rows) {
  if (tokens < 0 || top_k < 1 || rows < 0) return bad("tokens and rows must be >= 0, top_k >= 1");
  if (top_k > 1024 || tokens > kMaxSize / top_k || rows > kMaxSize)
    return bad("top_k above 1024, or more than 2^30 slots or rows");
  return DG_OK;
}

dg_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DG_OK;
  if (e == cudaErrorInvalidConfiguration) {
    cudaGetLastError();
    return set_errorf(DG_ERR_UNSUPPORTED, "%s: more than 2^30 tiles or CTAs", what);
  }
  return set_cuda_error(e, what);
}

// Bytes of scratch for a dispatch that quantizes the tokens before it copies
// their rows; 0 where it quantizes row by row.  Each row quantized by itself
// does a token's work up to top_k times, which for large calls is the larger
// part (16384 tokens of 2048 to 139 thousand rows: 145 us, the tokens once 77;
// with the sort, 512 tokens to 4096 rows 11.9 us against 9.9, 256 to 2048 9.2
// either way).
int64_t dispatch_scratch(int64_t tokens, int64_t width, int64_t rows) {
  if (tokens <= 0 || rows < 2 * tokens || rows * width < (int64_t(1) << 23)) return 0;
  return tokens * (ceil_div(width, 16) * 16 + 4 * ceil_div(width, kFp8Block));
}

// Whether a product of M rows goes to launch_fp8_skinny.  Its time grows with
// the rounds of 64 weight rows over the SMs (smaller tiles where those are
// few) and with each 8 rows; the tensor-core kernel's does not up to 128 rows,
// and is longer with 1 x 128 blocks in B.  Measured in us, weights from HBM,
// few-rows kernel / tensor-core kernel:
//   8 rows: 4096 x 8192 8.8 / 13.0, 12288 x 4096 14.1 / 14.1, 28672 x 8192 37 / 45;
//   16 rows: 8192 x 8192 17.1 / 19.2, 9600 x 4096 (150 tiles) 11.2 / 13.5, 9792 x
//   4096 (153) 17.9 / 13.6, its 1 x 128 form 18.2 / 18.6;
//   32 rows: 2400 x 8192 10.7 / 12.2, 4096 x 4096 10.2 / 10.3, 4096 x 8192 15.5 /
//   13.3, 8960 x 1536 9.1 / 7.4, its 1 x 128 form 9.1 / 9.1.
bool few_rows(int64_t M, int64_t N, int64_t K, int block_rows_b, int sm_count) {
  const int64_t t64 = ceil_div(N, 64), t32 = ceil_div(N, 32);
  if (M <= 8) return true;
  if (block_rows_b == 1) return M <= 16 || (M <= 32 && t64 <= sm_count);
  if (M <= 16) return t64 <= sm_count;
  return M <= 32 && 2 * t64 < sm_count && (2 * t32 < sm_count || N * K <= (int64_t(1) << 24));
}
// The same for experts' rows, by their mean: an expert with more than 8, 16 or
// 32 reads its weights again, the more often the more tiles there are.  Rows
// each at random, us: 64 experts of 4096 x 2048, 2 rows each 74.8 / 77.2, 4 86.6 /
// 89.0, 8 119 / 91.7, 16 160 / 93.6; 8 of 2048 x 2048 (256 tiles of 64), 6 8.6 /
// 13.5, 8 11.5 / 10.1; 4 of 2048 x 2048 (128 tiles), 12 6.7 / 9.6, 16 11.0 / 9.1.
// (Many experts of short K gain less: 128 of 2048 x 768, 2 rows each 48.7 / 40.8.)
bool few_rows_each(int64_t count, int64_t rows, int64_t N, int64_t K, int sm_count) {
  if (count == 1) return few_rows(rows, N, K, kFp8Block, sm_count);
  const int64_t tiles = std::min(count, rows) * ceil_div(N, 64);
  const int64_t most = tiles <= sm_count ? 12 : tiles <= 2 * sm_count ? 6 : 4;
  return rows <= most * count;
}

void fill_context(Fp8Args* a, const CallContext& c) {
  a->status = c.status;
  a->timeout_ns = c.timeout_ns;
  a->sm_count = c.sm_count;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_quantize_fp8(int64_t rows, int64_t K, dg_dtype dtype_x, const void* X, int64_t ldx,
                          int block_rows, void* codes, int64_t ldq, float* scales, int64_t lds,
                          void* codes_t, int64_t ldqt, float* scales_t, int64_t ldst,
                          dg_stream_t stream) {
  clear_error();
  dg_status s = check_sizes(rows, K, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype_x))
    return set_errorf(DG_ERR_UNSUPPORTED, "X is F16 or BF16, not %d", static_cast<int>(dtype_x));
  if (block_rows != 1 && block_rows != kFp8Block) return bad("block_rows must be 1 or 128");
  if (rows == 0 || K == 0) return DG_OK;
  if (!codes && !codes_t) return bad("no output");
  if ((s = check_rows16("X", X, ldx, K)) != DG_OK) return s;
  if (codes && (s = check_fp8("the codes", codes, ldq, K, scales, lds)) != DG_OK) return s;
  if (codes_t &&
      (s = check_fp8("the transposed codes", codes_t, ldqt, rows, scales_t, ldst)) != DG_OK)
    return s;
  if (ceil_div(rows, kFp8Block) * ceil_div(K, kFp8Block) > INT32_MAX)
    return set_error(DG_ERR_UNSUPPORTED, "more than 2^31 tiles of 128 x 128");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (block_rows == 1 && !codes_t) {
    Fp8RowsJob j;
    j.bf16 = dtype_x == DG_BF16;
    j.X = X;
    j.ldx = ldx;
    j.rows = rows;
    j.K = K;
    j.codes = codes;
    j.ldq = ldq;
    j.scales = scales;
    j.lds = lds;
    return launched(launch_quantize_fp8_rows(j, st, c.sm_count), "quantization launch");
  }
  const Fp8TilesJob j = {dtype_x == DG_BF16, X,    ldx,     rows, K,        block_rows != 1, codes,
                         ldq,                scales, lds, codes_t, ldqt, scales_t, ldst};
  return launched(launch_quantize_fp8_tiles(j, st), "quantization launch");
}

dg_status dg_gemm_fp8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                      const float* scale_a, int64_t lds_a, const void* B, int64_t ldb,
                      const float* scale_b, int64_t lds_b, int block_rows_b, void* D,
                      dg_dtype dtype_d, int64_t ldd, const void* bias, float alpha, float beta,
                      dg_epilogue epilogue, dg_stream_t stream) {
  clear_error();
  dg_status s = check_sizes(M, N, K);
  if (s != DG_OK) return s;
  if (block_rows_b != 1 && block_rows_b != kFp8Block) return bad("block_rows_b must be 1 or 128");
  if (M == 0 || N == 0) return DG_OK;
  Fp8Args a{};
  if ((s = check_output(D, dtype_d, ldd, N, bias, alpha, beta, epilogue, &a.epi)) != DG_OK)
    return s;
  if (K > 0) {
    if ((s = check_fp8("A", A, lda, K, scale_a, lds_a)) != DG_OK) return s;
    if ((s = check_fp8("B", B, ldb, K, scale_b, lds_b)) != DG_OK) return s;
  }
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.mode = Fp8Mode::kDense;
  a.M = M;
  a.N = N;
  a.K = K;
  a.A = A;
  a.lda = lda;
  a.sa = scale_a;
  a.lds_a = lds_a;
  a.B = B;
  a.ldb = ldb;
  a.sb = scale_b;
  a.lds_b = lds_b;
  a.block_rows_b = block_rows_b;
  a.count = 1;
  a.D = D;
  a.dtype_d = dtype_d;
  a.ldd = ldd;
  a.bias = bias;
  a.alpha = alpha;
  a.beta = beta;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  fill_context(&a, c);
  // K == 0 (only the epilogue is left) has no operands to describe to TMA
  return launched(K == 0 || few_rows(M, N, K, block_rows_b, c.sm_count) ? launch_fp8_skinny(a)
                                                                       : launch_fp8_tc(a),
                  "kernel launch");
}

dg_status dg_gemm_fp8_grouped(int64_t count, int64_t rows, int64_t N, int64_t K, const void* A,
                              int64_t lda, const float* scale_a, int64_t lds_a, const void* B,
                              int64_t ldb, int64_t stride_b, const float* scale_b, int64_t lds_b,
                              int64_t stride_sb, const int32_t* offsets, void* D,
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
  Fp8Args a{};
  if ((s = check_output(D, dtype_d, ldd, N, bias, alpha, beta, epilogue, &a.epi)) != DG_OK)
    return s;
  if (!offsets || !aligned4(offsets)) return bad("offsets is null or not 4-byte aligned");
  if (K > 0) {
    if ((s = check_fp8("A", A, lda, K, scale_a, lds_a)) != DG_OK) return s;
    if ((s = check_fp8("B", B, ldb, K, scale_b, lds_b)) != DG_OK) return s;
    if (count > 1 && (stride_b % ldb != 0 || stride_b / ldb < N))
      return bad("stride_b must be a multiple of ldb and at least N * ldb");
    if (count > 1 && stride_sb < ceil_div(N, kFp8Block) * lds_b)
      return bad("stride_sb must be at least ceil(N / 128) * lds_b");
    if ((count - 1) * (stride_b / ldb) + N > INT32_MAX)
      return set_error(DG_ERR_UNSUPPORTED, "more than 2^31 rows of weights");
  }
  if ((a.epi & kEpiBias) && stride_bias < 0) return bad("negative stride_bias");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.mode = Fp8Mode::kRows;
  a.M = rows;
  a.N = N;
  a.K = K;
  a.A = A;
  a.lda = lda;
  a.sa = scale_a;
  a.lds_a = lds_a;
  a.B = B;
  a.ldb = ldb;
  a.stride_b = count > 1 ? stride_b : N * ldb;
  a.sb = scale_b;
  a.lds_b = lds_b;
  a.stride_sb = count > 1 ? stride_sb : 0;
  a.block_rows_b = kFp8Block;
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
  fill_context(&a, c);
  return launched(K == 0 || few_rows_each(count, rows, N, K, c.sm_count) ? launch_fp8_skinny(a)
                                                                         : launch_fp8_tc(a),
                  "kernel launch");
}

dg_status dg_gemm_fp8_grouped_wgrad(int64_t count, int64_t M, int64_t N, int64_t rows,
                                    const void* A, int64_t lda, const float* scale_a,
                                    int64_t lds_a, const void* B, int64_t ldb,
                                    const float* scale_b, int64_t lds_b, const int32_t* offsets,
                                    void* D, dg_dtype dtype_d, int64_t ldd, int64_t stride_d,
                                    float alpha, float beta, dg_stream_t stream) {
  clear_error();
  dg_status s = check_sizes(M, N, rows);
  if (s != DG_OK) return s;
  if (count < 0) return bad("negative count");
  if (count > kMaxExperts)
    return set_errorf(DG_ERR_UNSUPPORTED, "more than %lld experts", (long long)kMaxExperts);
  if (count == 0 || M == 0 || N == 0) return DG_OK;
  Fp8Args a{};
  if ((s = check_output(D, dtype_d, ldd, N, nullptr, alpha, beta, DG_EPI_NONE, &a.epi)) != DG_OK)
    return s;
  if (count > 1 && stride_d < (M - 1) * ldd + N)
    return bad("stride_d is too small: the experts' gradients overlap");
  if (rows > 0) {
    if (!offsets || !aligned4(offsets)) return bad("offsets is null or not 4-byte aligned");
    if ((s = check_fp8("A", A, lda, rows, scale_a, lds_a)) != DG_OK) return s;
    if ((s = check_fp8("B", B, ldb, rows, scale_b, lds_b)) != DG_OK) return s;
  }
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  a.mode = rows > 0 ? Fp8Mode::kK : Fp8Mode::kDense;
  a.M = M;
  a.N = N;
  a.K = rows;
  a.A = A;
  a.lda = lda;
  a.sa = scale_a;
  a.lds_a = lds_a;
  a.B = B;
  a.ldb = ldb;
  a.sb = scale_b;
  a.lds_b = lds_b;
  a.block_rows_b = 1;
  a.count = count;
  a.offsets = offsets;
  a.D = D;
  a.dtype_d = dtype_d;
  a.ldd = ldd;
  a.stride_d = count > 1 ? stride_d : 0;
  a.alpha = alpha;
  a.beta = beta;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  fill_context(&a, c);
  if (rows > 0) return launched(launch_fp8_tc(a), "kernel launch");
  // no rows at all: every gradient is beta * D
  for (int64_t e = 0; e < count; ++e) {
    Fp8Args one = a;
    one.D = static_cast<uint8_t*>(D) + e * a.stride_d * (dtype_d == DG_F32 ? 4 : 2);
    if ((s = launched(launch_fp8_skinny(one), "kernel launch")) != DG_OK) return s;
  }
  return DG_OK;
}

int64_t dg_moe_rows(int64_t tokens, int64_t top_k, int64_t count, int64_t align) {
  if (check_routing(tokens, top_k, 0) != DG_OK || count < 1 || align < 1 || align > 1024) return -1;
  const int64_t slots = tokens * top_k;
  return ceil_div(slots + std::min(count, slots) * (align - 1), align) * align;
}

dg_status dg_moe_sort(int64_t tokens, int64_t top_k, int64_t count, const int32_t* ids,
                      int64_t align, int64_t rows, int32_t* offsets, int32_t* row_slot,
                      int32_t* slot_row, dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s != DG_OK) return s;
  if (count < 1) return bad("count must be >= 1");
  if (count > kMaxExperts)
    return set_errorf(DG_ERR_UNSUPPORTED, "more than %lld experts", (long long)kMaxExperts);
  if (align < 1 || align > 1024 || (align & (align - 1)) != 0)
    return bad("align must be a power of two up to 1024");
  const int64_t need = dg_moe_rows(tokens, top_k, count, align);
  if (rows < need)
    return set_errorf(DG_ERR_INVALID_ARG, "%lld rows, the sort may need %lld", (long long)rows,
                      (long long)need);
  if (!offsets || (tokens > 0 && (!ids || !slot_row)) || (rows > 0 && !row_slot))
    return bad("ids, offsets, row_slot or slot_row is null");
  if (!aligned4(ids) || !aligned4(offsets) || !aligned4(row_slot) || !aligned4(slot_row))
    return bad("ids, offsets, row_slot and slot_row must be 4-byte aligned");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  const MoeSortJob j = {tokens, top_k, count, ids, align, rows, offsets, row_slot, slot_row};
  return launched(launch_moe_sort(j, reinterpret_cast<cudaStream_t>(stream)), "sort launch");
}

dg_status dg_moe_dispatch(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                          const void* X, int64_t ldx, int64_t rows, const int32_t* row_slot,
                          void* D, int64_t ldd, dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype)) return set_error(DG_ERR_UNSUPPORTED, "rows are F16 or BF16");
  if (rows == 0 || width == 0) return DG_OK;
  if (!row_slot || !aligned4(row_slot)) return bad("row_slot is null or not 4-byte aligned");
  if (tokens > 0 && (s = check_rows16("X", X, ldx, width)) != DG_OK) return s;
  if ((s = check_rows16("D", D, ldd, width)) != DG_OK) return s;
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  MoeRowsJob j{};
  j.bf16 = dtype == DG_BF16;
  j.tokens = tokens;
  j.top_k = top_k;
  j.width = width;
  j.rows = rows;
  j.X = X;
  j.ldx = ldx;
  j.row_slot = row_slot;
  j.D = D;
  j.ldd = ldd;
  return launched(launch_moe_dispatch(j, reinterpret_cast<cudaStream_t>(stream), c.sm_count),
                  "dispatch launch");
}

int64_t dg_moe_dispatch_fp8_scratch(int64_t tokens, int64_t top_k, int64_t width, int64_t rows) {
  clear_error();
  if (check_routing(tokens, top_k, rows) != DG_OK || check_sizes(width, 0, 0) != DG_OK) return -1;
  return dispatch_scratch(tokens, width, rows);
}

dg_status dg_moe_dispatch_fp8(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                              const void* X, int64_t ldx, int64_t rows, const int32_t* row_slot,
                              void* codes, int64_t ldq, float* scales, int64_t lds,
                              dg_stream_t stream) {
  return dg_moe_dispatch_fp8_ex(tokens, top_k, width, dtype, X, ldx, rows, row_slot, codes, ldq,
                                scales, lds, nullptr, 0, stream);
}

dg_status dg_moe_dispatch_fp8_ex(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                                 const void* X, int64_t ldx, int64_t rows,
                                 const int32_t* row_slot, void* codes, int64_t ldq, float* scales,
                                 int64_t lds, void* scratch, int64_t scratch_bytes,
                                 dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype)) return set_error(DG_ERR_UNSUPPORTED, "rows are F16 or BF16");
  if (rows == 0 || width == 0) return DG_OK;
  if (!row_slot || !aligned4(row_slot)) return bad("row_slot is null or not 4-byte aligned");
  if (tokens > 0 && (s = check_rows16("X", X, ldx, width)) != DG_OK) return s;
  if ((s = check_fp8("the codes", codes, ldq, width, scales, lds)) != DG_OK) return s;
  const int64_t need = scratch ? dispatch_scratch(tokens, width, rows) : 0;
  if (scratch && !aligned16(scratch)) return bad("the scratch is not 16-byte aligned");
  if (scratch_bytes < need)
    return set_errorf(DG_ERR_INVALID_ARG, "%lld bytes of scratch, need %lld",
                      (long long)scratch_bytes, (long long)need);
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  Fp8RowsJob j;
  j.bf16 = dtype == DG_BF16;
  j.X = X;
  j.ldx = ldx;
  j.rows = rows;
  j.K = width;
  j.codes = codes;
  j.ldq = ldq;
  j.scales = scales;
  j.lds = lds;
  j.row_slot = row_slot;
  j.top_k = top_k;
  j.tokens = tokens;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (need > 0) {
    const int64_t pitch = ceil_div(width, 16) * 16, blocks = ceil_div(width, kFp8Block);
    Fp8RowsJob q = j;
    q.rows = tokens;
    q.codes = scratch;
    q.ldq = pitch;
    q.scales = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + tokens * pitch);
    q.lds = blocks;
    q.row_slot = nullptr;
    const cudaError_t e = launch_quantize_fp8_rows(q, st, c.sm_count);
    if (e != cudaSuccess) return launched(e, "dispatch launch");
    return launched(launch_moe_dispatch_codes(j, q.codes, pitch, q.scales, st, c.sm_count),
                    "dispatch launch");
  }
  return launched(launch_quantize_fp8_rows(j, st, c.sm_count), "dispatch launch");
}

dg_status dg_moe_combine(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                         const void* Y, int64_t ldy, int64_t rows, const int32_t* slot_row,
                         const float* weights, void* D, int64_t ldd, dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype)) return set_error(DG_ERR_UNSUPPORTED, "rows are F16 or BF16");
  if (tokens == 0 || width == 0) return DG_OK;
  if (!slot_row || !aligned4(slot_row)) return bad("slot_row is null or not 4-byte aligned");
  if (!aligned4(weights)) return bad("weights is not 4-byte aligned");
  if (rows > 0 && (s = check_rows16("Y", Y, ldy, width)) != DG_OK) return s;
  if ((s = check_rows16("D", D, ldd, width)) != DG_OK) return s;
  if (tokens * ceil_div(width, 8) / 256 >= INT32_MAX)
    return set_error(DG_ERR_UNSUPPORTED, "more than 2^31 CTAs");
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  MoeRowsJob j{};
  j.bf16 = dtype == DG_BF16;
  j.tokens = tokens;
  j.top_k = top_k;
  j.width = width;
  j.rows = rows;
  j.Y = Y;
  j.ldy = ldy;
  j.slot_row = slot_row;
  j.weights = weights;
  j.D = D;
  j.ldd = ldd;
  return launched(launch_moe_combine(j, reinterpret_cast<cudaStream_t>(stream)), "combine launch");
}

dg_status dg_moe_combine_backward(int64_t tokens, int64_t top_k, int64_t width, dg_dtype dtype,
                                  const void* dD, int64_t lddd, const void* Y, int64_t ldy,
                                  int64_t rows, const int32_t* row_slot, const int32_t* slot_row,
                                  const float* weights, void* dY, int64_t lddy, float* dweights,
                                  dg_stream_t stream) {
  clear_error();
  dg_status s = check_routing(tokens, top_k, rows);
  if (s == DG_OK) s = check_sizes(width, 0, 0);
  if (s != DG_OK) return s;
  if (!type16(dtype)) return set_error(DG_ERR_UNSUPPORTED, "rows are F16 or BF16");
  if (tokens == 0 && rows == 0) return DG_OK;
  if ((rows > 0 && !row_slot) || (tokens > 0 && !slot_row))
    return bad("row_slot or slot_row is null");
  if (!aligned4(row_slot) || !aligned4(slot_row) || !aligned4(weights) || !aligned4(dweights))
    return bad("row_slot, slot_row, weights and dweights must be 4-byte aligned");
  if (tokens > 0 && width > 0 && (s = check_rows16("dD", dD, lddd, width)) != DG_OK) return s;
  if (rows > 0 && width > 0) {
    if ((s = check_rows16("dY", dY, lddy, width)) != DG_OK) return s;
    if (dweights && (s = check_rows16("Y", Y, ldy, width)) != DG_OK) return s;
  }
  CallContext c;
  if ((s = call_context(&c)) != DG_OK) return s;
  MoeRowsJob j{};
  j.bf16 = dtype == DG_BF16;
  j.tokens = tokens;
  j.top_k = top_k;
  j.width = width;
  j.rows = rows;
  j.X = dD;
  j.ldx = lddd;
  j.Y = Y;
  j.ldy = ldy;
  j.row_slot = row_slot;
  j.slot_row = slot_row;
  j.weights = weights;
  j.D = dY;
  j.ldd = lddy;
  j.dweights = dweights;
  return launched(launch_moe_combine_backward(j, reinterpret_cast<cudaStream_t>(stream)),
                  "combine gradient launch");
}

}  // extern "C"
