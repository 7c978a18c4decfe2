// Pieces shared by the FP8 (E4M3 with block scales) and expert-routing
// kernels: 16-bit loads as FP32, block scales, conversions and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dg {
namespace fp8 {

constexpr int kBlock = 128;              // values per scale along K
constexpr float kTop = 448.0f;           // largest finite E4M3 value
constexpr float kFloor = 448.0f * 0x1p-126f;  // a block's amax is taken as at least this

// The two 16-bit floating types behind one interface.
struct F16 {
  static constexpr uint32_t kInf = 0x7C00u;  // magnitudes from here on are infinite or NaN
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float one(uint32_t h) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
  }
};
struct BF16 {
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float one(uint32_t h) { return __uint_as_float(h << 16); }
};

// Four FP32 values -> four E4M3 codes (v0 in the low byte), nearest, ties to
// even, saturated to the largest finite value.
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return out;
}

// Quotients rounded to nearest, for a in [kFloor, 2^100): the quotient by an
// approximate reciprocal, corrected by its remainder, which one FMA gives
// exactly (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, 1990).  The general division takes a tenth of the row
// kernel's time.
__device__ __forceinline__ float over_top(float a) {  // a / 448
  constexpr float c = 1.0f / kTop;
  const float q = a * c;
  return fmaf(fmaf(-q, kTop, a), c, q);
}
__device__ __forceinline__ float top_over(float a) {  // 448 / a
  float f;
  asm("rcp.approx.f32 %0, %1;" : "=f"(f) : "f"(a));
  f = fmaf(fmaf(-a, f, 1.0f), f, f);
  const float q = kTop * f;
  return fmaf(fmaf(-q, a, kTop), f, q);
}

// What quantizes a block: its scale and the factor that its values take.  A
// block with an infinity or a NaN has the scale NaN and codes 0.
struct BlockScale {
  float scale, factor;
  bool bad;
};
template <typename T>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  BlockScale b;
  b.bad = amax_bits >= T::kInf;
  const float amax = fmaxf(T::one(b.bad ? 0u : amax_bits), kFloor);
  b.factor = top_over(amax);
  b.scale = over_top(amax);
  if (amax >= 0x1p100f) {  // the reciprocal nears the subnormal range
    b.factor = __fdiv_rn(kTop, amax);
    b.scale = __fdiv_rn(amax, kTop);
  }
  if (b.bad) b.scale = CUDART_NAN_F;
  return b;
}

// Eight 16-bit values (four words) -> eight codes.
template <typename T>
__device__ __forceinline__ uint2 quantize8(const uint32_t (&w)[4], const BlockScale& b) {
  if (b.bad) return make_uint2(0u, 0u);
  const float2 x0 = T::unpack(w[0]), x1 = T::unpack(w[1]), x2 = T::unpack(w[2]),
               x3 = T::unpack(w[3]);
  const float f = b.factor;
  return make_uint2(e4m3x4(x0.x * f, x0.y * f, x1.x * f, x1.y * f),
                    e4m3x4(x2.x * f, x2.y * f, x3.x * f, x3.y * f));
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return d;
}

// GELU of two values: t Phi(t) = max(t, 0) + b Phi(b), b = -|t|, with Phi the
// normal distribution function and Phi(b) = 2^P(b).  P(b) = -1 + b R(b) is a
// weighted least-squares fit of log2 Phi on [-6, 0], reweighted until the errors
// of Phi were level: at most 1.0e-7, and 2.2e-4 of Phi there; P falls steadily
// below -6 (an error of 3e-12 of GELU) and is cut off at -16, for infinities.
// The GELU of a tile costs as much as several of its K blocks: one exponential
// per value and eight packed FMAs per two, without the reciprocal that the
// form with exp(-t^2 / 2) times a polynomial takes (both share the unit of 16
// results per clock and SM).
__device__ __forceinline__ float2 gelu2(float2 t) {
  constexpr float c[9] = {-1.0f,           1.15111136f,     -4.59140331e-1f,
                          5.27343079e-2f,  7.43800076e-3f,  4.35754948e-4f,
                          -6.15835597e-5f, -1.36701265e-5f, -7.71337284e-7f};
  float2 b, m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(b.x) : "f"(-fabsf(t.x)), "f"(-16.0f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(b.y) : "f"(-fabsf(t.y)), "f"(-16.0f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.x) : "f"(t.x), "f"(0.0f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.y) : "f"(t.y), "f"(0.0f));
  float2 q = make_float2(c[8], c[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) q = fma2(q, b, make_float2(c[i], c[i]));
  return fma2(b, make_float2(ex2_approx(q.x), ex2_approx(q.y)), m);
}

}  // namespace fp8
}  // namespace dg
