// Block quantization of FP16 / BF16 rows to 4-bit codes with an E4M3 scale per
// 16 values and an FP32 scale per row (dg_quantize_nvf4), the same on rows
// gathered by expert (dg_moe_dispatch_nvf4), and the way back
// (dg_dequantize_nvf4).
//
// Row scale r = the smallest power of two with 2688 r >= the row's largest
// magnitude (2688 = 6 * 448: then no block's scale leaves E4M3), or the
// caller's.  Per block of 16, every quotient and product rounded to FP32:
//   scale = max(e4m3(amax / (6 r)), 2^-9),  code = e2m1(v / (scale * r)).
// A power of two costs no precision (E4M3 has the same relative step
// everywhere) and needs no division for r.  What matters of a quotient is that a
// value in the middle between two codes is found there; another is at least 2^-12
// away.  With a power of two for r the divisor has 4 significant bits and a middle
// 3, and products by the reciprocal find every one: for scales with 1 / 6 rounded to
// nearest, for codes with the reciprocal rounded up and the product towards zero (of 15
// times 7 combinations none is missed; with products to nearest, 14 are.  Tests enumerate
// them in exact arithmetic, and every scale with every middle on the GPU, at row scales
// from 2^-100 to 2^116).  With the caller's r the quotients are corrected by their
// remainders.
//
// Scales leave in the tiles that the tensor core's scale copies read: 128 rows
// x 4 blocks in 512 bytes, line l (16 bytes) holding rows l, 32 + l, 64 + l and
// 96 + l, four bytes each.  So neighbours in the work are a line's four rows.
//
// Bound by memory: 2 bytes read, 0.56 written per value.  A row is read once:
// 2^log2_tpr threads share it and hold it, 16 values x kGroups each, while its
// largest magnitude is found (rows of more than 16384 values are read again,
// from L2).  8192 x 4096 BF16: quantization 19.2 us (4.5 TB/s; with 32 values a thread
// 25.1), with given row scales 24.1, the way back 16.8 us, its stores at 4.0 TB/s, what
// clearing a buffer reaches.
#include <algorithm>

#include <cuda_runtime.h>

#include "convert.cuh"
#include "fp8.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kThreads = 256;
constexpr int kGroup = 16;   // values per scale
constexpr int kGroups = 4;   // held by a thread
constexpr int kMinExp = -100;  // of a row scale

struct QuantParams {
  const uint16_t* X;
  int64_t ldx, stride_x;
  int64_t rows, K, rows_pad, total;  // total = count * rows_pad
  int nblk, nblk_pad, log2_tpr;
  uint8_t* codes;
  int64_t ldq, stride_q;
  uint8_t* scales;
  float* row_scales;
  const float* given;
  const int32_t* row_slot;  // gather: row r is X's row row_slot[r] / top_k
  int top_k;
  int64_t tokens;
};

// 16 consecutive values as 8 words, zeros past n.  Once: they are not read again (8191
// x 4096 there and back 37.1 us, without the hint 38.0).
template <bool Once>
__device__ __forceinline__ void load16(const uint16_t* p, int64_t n, uint32_t (&w)[8]) {
  if (n >= 16) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
    const uint4 a = Once ? __ldcs(v) : __ldg(v), b = Once ? __ldcs(v + 1) : __ldg(v + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = 2 * i < n ? p[2 * i] : 0u;
      const uint32_t hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
      w[i] = lo | (hi << 16);
    }
  }
}

__device__ __forceinline__ uint32_t amax_bits16(const uint32_t (&w)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// The smallest power of two r >= 2^kMinExp with 2688 r >= amax.
__device__ __forceinline__ float row_scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // 2688 = 1.3125 * 2^11: a mantissa above 0.3125 needs the next exponent
  const int e = static_cast<int>(b >> 23) - 127 - 11 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, kMinExp) + 127) << 23);
}

// One nonnegative value as E4M3, nearest, ties to even, saturated.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(v));
  return two & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  return F16::one(h & 0xFFFFu);
}

__device__ __forceinline__ float2 mul2_rz(float2 a, float2 b) {
  float2 d;
  asm("mul.rz.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return d;
}

// Codes of a block of 16 (two words) and its scale byte.  d6 = 6 r and its
// reciprocal.  Given: quotients by a reciprocal corrected by the remainder, which
// one FMA gives exactly (P. Markstein, Computation of elementary functions on the
// IBM RISC System/6000 processor, 1990).
template <typename T, bool Given>
__device__ __forceinline__ uint2 quantize16(const uint32_t (&w)[8], uint32_t amax_bits, float r,
                                            float d6, float d6_inv, uint32_t& byte) {
  if (amax_bits >= T::kInf) {
    byte = 0x7Fu;  // NaN
    return make_uint2(0u, 0u);
  }
  const float amax = T::one(amax_bits);
  float t = amax * d6_inv;
  if (Given) {
    t = fmaf(fmaf(-t, d6, amax), d6_inv, t);
    t = amax >= 512.0f * d6 ? 448.0f : t;  // the quotient may have overflowed
  }
  byte = max(e4m3_of(t), 1u);
  const float u = e4m3_value(byte) * r;
  const float f = Given ? __frcp_rn(u) : __frcp_ru(u);
  const float2 f2 = make_float2(f, f), u2 = make_float2(-u, -u);
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x = T::unpack(w[4 * h + i]);
      if (!Given) {
        x = mul2_rz(x, f2);
        v[2 * i] = x.x;
        v[2 * i + 1] = x.y;
      } else {
        // beyond 8 u every code is the largest one
        x.x = fminf(fmaxf(x.x, -8.0f * u), 8.0f * u);
        x.y = fminf(fmaxf(x.y, -8.0f * u), 8.0f * u);
        float2 q = mul2(x, f2);
        q = fma2(fma2(q, u2, x), f2, q);
        // the sign of a zero, which the correction loses
        v[2 * i] = copysignf(q.x, x.x);
        v[2 * i + 1] = copysignf(q.y, x.y);
      }
    }
    o[h] = e2m1x8_from_f32(v);
  }
  return make_uint2(o[0], o[1]);
}

template <typename T, bool Gather, bool Given>
__global__ void __launch_bounds__(kThreads, Given ? 3 : 4)
    quantize_nvf4_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t red[2][kThreads / 32];
  grid_dependency_wait();  // launched as a dependent of the previous kernel
  grid_launch_dependents();
  const int tpr = 1 << p.log2_tpr;
  const int t = threadIdx.x & (tpr - 1);
  const int rows_per_pass = kThreads >> p.log2_tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_pass;
  const int chunk = tpr * kGroups;
  int turn = 0;
  // (128 rows are a whole number of passes: every thread has a row, or a padding one)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_per_pass; base < p.total;
       base += step) {
    const int64_t at = base + (threadIdx.x >> p.log2_tpr);
    const int64_t z = p.total == p.rows_pad ? 0 : at / p.rows_pad, in = at - z * p.rows_pad;
    const int64_t tile = in >> 7;
    const int line = static_cast<int>(in >> 2) & 31, part = static_cast<int>(in) & 3;
    const int64_t row = tile * 128 + part * 32 + line;
    const bool there = row < p.rows;
    const uint16_t* src = nullptr;
    if (there) {
      if (Gather) {
        const int slot = __ldg(p.row_slot + row);
        const int64_t token = slot < 0 ? -1 : static_cast<int64_t>(slot / p.top_k);
        if (token >= 0 && token < p.tokens) src = p.X + token * p.ldx;
      } else {
        src = p.X + z * p.stride_x + row * p.ldx;
      }
    }
    uint32_t w[kGroups][8], m[kGroups];
    uint32_t most = 0;
    auto load = [&](int c0) {
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const int g = c0 + j * tpr + t;
        const int64_t n = p.K - static_cast<int64_t>(g) * kGroup;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[j][i] = 0u;
        if (src && n > 0) load16<!Gather>(src + static_cast<int64_t>(g) * kGroup, n, w[j]);
      }
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        m[j] = amax_bits16(w[j]);
        if (m[j] < T::kInf) most = max(most, m[j]);
      }
    };
    // (the last chunk stays in the registers; of several, all are read again)
    for (int c0 = 0; c0 < p.nblk; c0 += chunk) load(c0);
    float r;
    bool odd = false;
    if (Given) {
      r = there ? __ldg(p.given + z * p.rows + row) : 1.0f;
      odd = !(r >= 0x1p-100f && r <= 0x1p100f);
      if (odd) r = 1.0f;
    } else {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
        if (d < tpr) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
      if (tpr > 32) {
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = most;
        // the row's own barrier (with the CTA's, 8191 x 4096 took 0.7 us longer)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (threadIdx.x >> p.log2_tpr)), "r"(tpr) : "memory");
        const int first = (threadIdx.x >> 5) & ~((tpr >> 5) - 1);
        for (int i = 0; i < tpr >> 5; ++i) most = max(most, red[turn][first + i]);
        turn ^= 1;  // (a buffer is written again only after the next barrier)
      }
      r = row_scale_for(T::one(most));
      if (there && t == 0) p.row_scales[z * p.rows + row] = r;
    }
    const float d6 = 6.0f * r, d6_inv = __frcp_rn(d6);
    uint8_t* qrow = p.codes + z * p.stride_q + row * p.ldq;
    uint8_t* tiles = p.scales + (z * (p.rows_pad >> 7) + tile) * (p.nblk_pad >> 2) * 512 +
                     line * 16 + part * 4;
    for (int c0 = 0; c0 < p.nblk; c0 += chunk) {
      if (p.nblk > chunk) load(c0);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const int g = c0 + j * tpr + t;
        uint32_t byte = 0;
        if (there && g < p.nblk) {
          const uint2 q = quantize16<T, Given>(w[j], odd ? T::kInf : m[j], r, d6, d6_inv, byte);
          uint8_t* dst = qrow + static_cast<int64_t>(g) * 8;
          const int64_t n = p.K - static_cast<int64_t>(g) * kGroup;
          if (n >= kGroup) {
            *reinterpret_cast<uint2*>(dst) = q;
          } else {
            const int bytes = static_cast<int>((n + 1) / 2);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < bytes)
                dst[i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
          }
        }
        uint32_t word = byte << (8 * (t & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        if ((t & 3) == 0 && g < p.nblk_pad)
          *reinterpret_cast<uint32_t*>(tiles + static_cast<int64_t>(g >> 2) * 512) = word;
      }
    }
  }
}

template <typename T>
cudaError_t run_quantize(const Nvf4RowsJob& j, const QuantParams& p, int grid,
                         cudaStream_t stream) {
  const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
  if (j.row_slot) return launch_dependent(quantize_nvf4_kernel<T, true, false>, g, b, 0, stream, p);
  if (j.given) return launch_dependent(quantize_nvf4_kernel<T, false, true>, g, b, 0, stream, p);
  return launch_dependent(quantize_nvf4_kernel<T, false, false>, g, b, 0, stream, p);
}

// ---------------------------------------------------------------------------
// The way back: value = e2m1(code) * (scale * r), a thread per block of 16.
// ---------------------------------------------------------------------------
struct ValuesParams {
  const uint8_t* codes;
  int64_t ldq, stride_q;
  const uint8_t* scales;
  const float* row_scales;
  void* D;
  int64_t ldd, stride_d;
  int64_t rows, K, total;  // total = count * rows * nblk
  int nblk, tiles_k, tiles_m, dtype_d, vec, one;  // one: a single matrix
};

template <int Bytes>
__device__ __forceinline__ void store_values(void* d, const float (&v)[16], int64_t n, bool vec,
                                             bool bf16) {
  uint32_t w[4 * Bytes];
#pragma unroll
  for (int i = 0; i < 4 * Bytes; ++i)
    w[i] = Bytes == 4 ? __float_as_uint(v[i])
                      : bf16 ? BF16::pack(v[(2 * i) & 15], v[(2 * i + 1) & 15])
                             : F16::pack(v[(2 * i) & 15], v[(2 * i + 1) & 15]);
  if (vec && n >= kGroup) {
#pragma unroll
    for (int i = 0; i < Bytes; ++i)
      static_cast<uint4*>(d)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (i < n) {
        if (Bytes == 4)
          static_cast<uint32_t*>(d)[i] = w[i];
        else
          static_cast<uint16_t*>(d)[i] = static_cast<uint16_t>(w[(i >> 1) & (4 * Bytes - 1)] >> (16 * (i & 1)));
      }
  }
}

__global__ void __launch_bounds__(kThreads)
    dequantize_nvf4_kernel(const __grid_constant__ ValuesParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.total;
       i += step) {
    // (64-bit divisions only where they are needed: 8192 x 4096 16.7 us with them)
    const int64_t flat = p.total <= UINT32_MAX ? static_cast<uint32_t>(i) / static_cast<uint32_t>(p.nblk)
                                               : i / p.nblk;
    const int g = static_cast<int>(i - flat * p.nblk);
    const int64_t z = p.one ? 0 : flat / p.rows, row = flat - z * p.rows;
    const int64_t n = p.K - static_cast<int64_t>(g) * kGroup;
    const uint8_t* src = p.codes + z * p.stride_q + row * p.ldq + static_cast<int64_t>(g) * 8;
    uint32_t c[2] = {0u, 0u};
    if (n >= kGroup) {
      const uint2 q = *reinterpret_cast<const uint2*>(src);
      c[0] = q.x, c[1] = q.y;
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (2 * b < n) c[b >> 2] |= static_cast<uint32_t>(src[b]) << (8 * (b & 3));
    }
    const int64_t tile = (z * p.tiles_m + (row >> 7)) * p.tiles_k + (g >> 2);
    const uint32_t s = p.scales[tile * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (g & 3)];
    const float u = e4m3_value(s) * p.row_scales[flat];
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[4];
      e2m1x8_to_f16x2x4(c[h], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = F16::unpack(f[k]);
        v[8 * h + 2 * k] = x.x * u;
        v[8 * h + 2 * k + 1] = x.y * u;
      }
    }
    const int64_t d = z * p.stride_d + row * p.ldd + static_cast<int64_t>(g) * kGroup;
    if (p.dtype_d == DG_F32)
      store_values<4>(static_cast<uint32_t*>(p.D) + d, v, n, p.vec, false);
    else
      store_values<2>(static_cast<uint16_t*>(p.D) + d, v, n, p.vec, p.dtype_d == DG_BF16);
  }
}

}  // namespace

cudaError_t launch_quantize_nvf4(const Nvf4RowsJob& j, cudaStream_t stream, int sm_count) {
  QuantParams p;
  p.X = static_cast<const uint16_t*>(j.X);
  p.ldx = j.ldx;
  p.stride_x = j.stride_x;
  p.rows = j.rows;
  p.K = j.K;
  p.rows_pad = (j.rows + 127) / 128 * 128;
  p.total = j.count * p.rows_pad;
  p.nblk = static_cast<int>((j.K + kGroup - 1) / kGroup);
  p.nblk_pad = (p.nblk + 3) / 4 * 4;
  p.codes = static_cast<uint8_t*>(j.codes);
  p.ldq = j.ldq;
  p.stride_q = j.stride_q;
  p.scales = static_cast<uint8_t*>(j.scales);
  p.row_scales = j.row_scales;
  p.given = j.given;
  p.row_slot = j.row_slot;
  p.top_k = static_cast<int>(j.top_k);
  p.tokens = j.tokens;
  // the fewest threads (at least a quad, for the scale words) that hold a row;
  // more where that leaves SMs without work
  int log2_tpr = 2;
  while (log2_tpr < 8 && (kGroups << log2_tpr) < p.nblk_pad) ++log2_tpr;
  while (log2_tpr < 8 && (1 << log2_tpr) < p.nblk_pad &&
         (p.total << log2_tpr) / kThreads < 4 * sm_count)
    ++log2_tpr;
  p.log2_tpr = log2_tpr;
  const int64_t passes = p.total / (kThreads >> log2_tpr);
  const int grid = static_cast<int>(std::min<int64_t>(passes, int64_t(sm_count) * 16));
  const cudaError_t e =
      j.bf16 ? run_quantize<BF16>(j, p, grid, stream) : run_quantize<F16>(j, p, grid, stream);
  count_launches(1);
  return e;
}

cudaError_t launch_dequantize_nvf4(const Nvf4ValuesJob& j, cudaStream_t stream, int sm_count) {
  ValuesParams p;
  p.codes = static_cast<const uint8_t*>(j.codes);
  p.ldq = j.ldq;
  p.stride_q = j.stride_q;
  p.scales = static_cast<const uint8_t*>(j.scales);
  p.row_scales = j.row_scales;
  p.D = j.D;
  p.ldd = j.ldd;
  p.stride_d = j.stride_d;
  p.rows = j.rows;
  p.K = j.K;
  p.nblk = static_cast<int>((j.K + kGroup - 1) / kGroup);
  p.tiles_k = (p.nblk + 3) / 4;
  p.tiles_m = static_cast<int>((j.rows + 127) / 128);
  p.total = j.count * j.rows * p.nblk;
  p.dtype_d = static_cast<int>(j.dtype_d);
  p.one = j.count == 1 ? 1 : 0;
  const int64_t z = j.dtype_d == DG_F32 ? 4 : 2;
  p.vec = (reinterpret_cast<uintptr_t>(j.D) & 15) == 0 && (j.ldd * z) % 16 == 0 &&
                  (j.stride_d * z) % 16 == 0
              ? 1
              : 0;
  const int64_t ctas = (p.total + kThreads - 1) / kThreads;
  const int grid = static_cast<int>(std::min<int64_t>(ctas, int64_t(sm_count) * 32));
  const cudaError_t e = launch_dependent(dequantize_nvf4_kernel, dim3(static_cast<unsigned>(grid)),
                                         dim3(kThreads), 0, stream, p);
  count_launches(1);
  return e;
}

}  // namespace dg
