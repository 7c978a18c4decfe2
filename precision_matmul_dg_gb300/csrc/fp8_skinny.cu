// FP8 (E4M3) product with block scales for few rows (dg_gemm_fp8 with M <=
// 16, dg_gemm_fp8_grouped with few rows per expert):
//   D[m,n] = epilogue(alpha * sum over blocks b of sa[m,b] * sb[n,b] *
//            sum over k in b of A[m,k] * B[n,k] + beta * D[m,n])
//
// The job is to stream N * K bytes of weights; each is used M times.  The
// weights go from memory straight into registers as the 16-row operand of
// warp-level m16n8k32 E4M3 MMAs, the activations are the 8-column operand.
// The order of K inside a block is free as long as both operands share it, so
// a lane's fragments are 16-byte pieces of its rows: lane (g = lane / 4, q =
// lane % 4) holds bytes 64 h + 16 q .. + 15 of rows g and g + 8 for the two
// halves h of a 128-byte block, words 2 s and 2 s + 1 of a piece going to MMA
// step s.  Four MMAs make a block's sums, which then take the block's scales
// in FP32.
//
// A CTA's warps are 2^log2_slices slices of K by row groups of 16 weights;
// slice w takes blocks w, w + slices, ... and the slices' sums meet in shared
// memory in slice order (bit-stable).
#include <algorithm>

#include "epilogue.cuh"
#include "fp8.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnroll = 2;  // blocks in flight per warp: 4 x 16 bytes of weights per lane each

struct SkinnyParams {
  const uint8_t* A;
  int64_t lda;
  const float* sa;
  int64_t lds_a;
  const uint8_t* B;
  int64_t ldb, stride_b;
  const float* sb;
  int64_t lds_b, stride_sb;
  const int32_t* offsets;  // NULL: one product over M rows
  void* D;
  int64_t ldd;
  const void* bias;
  int64_t stride_bias;
  float alpha, beta;
  int M, N, K, flags, dtype_d, block_rows_b, log2_slices;
};

// c += a (16 x 32, weights) . b (32 x 8, activations)
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 16 bytes of a row at k, zeros from K on (k < K; a row's bytes up to K
// rounded up to 16 are there).
__device__ __forceinline__ uint4 mask16(uint4 v, int n) {
  if (n >= 16) return v;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    if (left < 4) w[i] = left <= 0 ? 0u : w[i] & (0xFFFFFFFFu >> (8 * (4 - left)));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == DG_F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == DG_BF16 ? BF16::one(h) : F16::one(h);
}

template <int NT>  // groups of 8 activation rows at a time
__global__ void __launch_bounds__(kThreads)
    skinny_fp8_kernel(const __grid_constant__ SkinnyParams p) {
  __shared__ float red[kWarps][NT * 4][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int slices = 1 << p.log2_slices;
  const int slice = warp & (slices - 1), group = warp >> p.log2_slices;
  const int groups = kWarps >> p.log2_slices;
  const int expert = blockIdx.y;
  const int n0 = (static_cast<int>(blockIdx.x) * groups + group) * 16;
  int row0 = 0, row1 = p.M;
  if (p.offsets) {
    row0 = min(max(__ldg(p.offsets + expert), 0), p.M);
    row1 = min(max(__ldg(p.offsets + expert + 1), 0), p.M);
  }
  const uint8_t* B = p.B + expert * p.stride_b;
  const float* sb = p.sb + expert * p.stride_sb;
  // weight rows past N: clamped, their results are not stored
  const int na = min(n0 + g, p.N - 1), nb = min(n0 + g + 8, p.N - 1);
  const uint8_t* wa = B + na * p.ldb;
  const uint8_t* wb = B + nb * p.ldb;
  const float* sba = sb + static_cast<int64_t>(na / p.block_rows_b) * p.lds_b;
  const float* sbb = sb + static_cast<int64_t>(nb / p.block_rows_b) * p.lds_b;
  const int blocks = (p.K + kBlock - 1) / kBlock;

  for (int m0 = row0; m0 < row1; m0 += 8 * NT) {
    float acc[NT][4];
    const uint8_t* xa[NT];
    const float* sx[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
      // activation rows past the last: clamped, their results are not stored
      xa[t] = p.A + static_cast<int64_t>(min(m0 + 8 * t + g, row1 - 1)) * p.lda;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sx[t][i] = p.sa + static_cast<int64_t>(min(m0 + 8 * t + 2 * q + i, row1 - 1)) * p.lds_a;
    }
    for (int b0 = slice; b0 < blocks; b0 += slices * kUnroll) {
      uint4 w[kUnroll][4];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = (b0 + u * slices) * kBlock + 16 * q;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kk = k + 64 * h;
          w[u][2 * h] = w[u][2 * h + 1] = make_uint4(0u, 0u, 0u, 0u);
          if (kk < p.K) {
            w[u][2 * h] = ld_stream16(wa + kk);
            w[u][2 * h + 1] = ld_stream16(wb + kk);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int b = b0 + u * slices;
        if (b >= blocks) break;
        const int k = b * kBlock + 16 * q;
        const float swa = __ldg(sba + b), swb = __ldg(sbb + b);
        if ((b + 1) * kBlock > p.K) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[u][i] = mask16(w[u][i], p.K - k - 64 * (i >> 1));
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (k + 64 * h < p.K)
              x = mask16(__ldg(reinterpret_cast<const uint4*>(xa[t] + k + 64 * h)),
                         p.K - k - 64 * h);
            const uint4 lo = w[u][2 * h], hi = w[u][2 * h + 1];
            mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
            mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
          }
          const float s0 = __ldg(sx[t][0] + b), s1 = __ldg(sx[t][1] + b);
          acc[t][0] = fmaf(c[0], s0 * swa, acc[t][0]);
          acc[t][1] = fmaf(c[1], s1 * swa, acc[t][1]);
          acc[t][2] = fmaf(c[2], s0 * swb, acc[t][2]);
          acc[t][3] = fmaf(c[3], s1 * swb, acc[t][3]);
        }
      }
    }
    if (slices > 1) {
      __syncthreads();  // the last round's sums have been read
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][4 * t + i][lane] = acc[t][i];
      __syncthreads();
      if (slice != 0) continue;
      for (int s = 1; s < slices; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] += red[warp + s][4 * t + i][lane];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + 8 * t + 2 * q + (i & 1), n = n0 + g + 8 * (i >> 1);
        if (m >= row1 || n >= p.N) continue;
        const int64_t at = m * p.ldd + n;
        float v = p.alpha * acc[t][i];
        if (p.beta != 0.0f) v = fmaf(p.beta, load_as_f32(p.D, at, p.dtype_d), v);
        if (p.flags & kEpiBias) v += load_as_f32(p.bias, expert * p.stride_bias + n, p.dtype_d);
        if (p.flags & kEpiGelu) v = gelu_erf(v);
        if (p.dtype_d == DG_F32)
          static_cast<float*>(p.D)[at] = v;
        else
          static_cast<uint16_t*>(p.D)[at] = static_cast<uint16_t>(
              p.dtype_d == DG_BF16 ? BF16::pack(v, 0.0f) : F16::pack(v, 0.0f));
      }
  }
}

}  // namespace

cudaError_t launch_fp8_skinny(const Fp8Args& a) {
  SkinnyParams p;
  p.A = static_cast<const uint8_t*>(a.A);
  p.lda = a.lda;
  p.sa = a.sa;
  p.lds_a = a.lds_a;
  p.B = static_cast<const uint8_t*>(a.B);
  p.ldb = a.ldb;
  p.stride_b = a.stride_b;
  p.sb = a.sb;
  p.lds_b = a.lds_b;
  p.stride_sb = a.stride_sb;
  p.offsets = a.mode == Fp8Mode::kRows ? a.offsets : nullptr;
  p.D = a.D;
  p.ldd = a.ldd;
  p.bias = a.bias;
  p.stride_bias = a.stride_bias;
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.flags = a.epi;
  p.dtype_d = static_cast<int>(a.dtype_d);
  p.block_rows_b = a.block_rows_b;
  const int64_t experts = p.offsets ? a.count : 1;
  const int64_t row_groups = (a.N + 15) / 16;
  // slices of K until the warps fill the SMs, at least one block each
  const int64_t blocks = (a.K + kBlock - 1) / kBlock;
  int log2_slices = 0;
  while (log2_slices < 3 && (2 << log2_slices) <= blocks &&
         ((row_groups * std::min(experts, a.M)) << log2_slices) < 16 * a.sm_count)
    ++log2_slices;
  p.log2_slices = log2_slices;
  const int64_t groups = kWarps >> log2_slices;
  const dim3 grid(static_cast<unsigned>((row_groups + groups - 1) / groups),
                  static_cast<unsigned>(experts));
  // eight activation rows at a time where most products have no more
  const int64_t rows_each = p.offsets ? (a.M + experts - 1) / experts : a.M;
  const cudaError_t e =
      rows_each <= 8
          ? launch_dependent(skinny_fp8_kernel<1>, grid, dim3(kThreads), 0, a.stream, p)
          : launch_dependent(skinny_fp8_kernel<2>, grid, dim3(kThreads), 0, a.stream, p);
  count_launches(1);
  return e;
}

}  // namespace dg
