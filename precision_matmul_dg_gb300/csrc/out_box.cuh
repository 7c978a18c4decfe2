// The way out of the 8-bit and 4-bit products on tcgen05: values converted to
// D's type, staged by a warp as a box of 32 rows x 128 bytes in shared memory,
// and sent to D by TMA or by the warp.
#pragma once

#include <stdint.h>

#include "fp8.cuh"
#include "tc_common.cuh"

namespace dg {
namespace fp8 {

constexpr int kBoxRow = 128, kBoxBytes = 32 * kBoxRow;  // a box of D: 32 rows of 128 bytes

// Lane 0's arrival, predicated instead of branched around.
__device__ __forceinline__ void lane0_arrive(uint32_t bar, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(lane)
      : "memory");
}

template <typename T>
__device__ __forceinline__ uint4 pack8(float2 a, float2 b, float2 c, float2 d) {
  return make_uint4(T::pack(a.x, a.y), T::pack(b.x, b.y), T::pack(c.x, c.y), T::pack(d.x, d.y));
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == DG_F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == DG_BF16 ? BF16::one(h) : F16::one(h);
}

// v[i] += k * (the 16 values of dtype from p on), the first n of them; 16-byte
// loads where there are 16 at such an address.
__device__ __forceinline__ void add16(float (&v)[16], float k, const void* p, int dtype, int n) {
  if (n >= 16 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const uint4* q = static_cast<const uint4*>(p);
    if (dtype == DG_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = q[i];
        v[4 * i] = fmaf(k, __uint_as_float(w.x), v[4 * i]);
        v[4 * i + 1] = fmaf(k, __uint_as_float(w.y), v[4 * i + 1]);
        v[4 * i + 2] = fmaf(k, __uint_as_float(w.z), v[4 * i + 2]);
        v[4 * i + 3] = fmaf(k, __uint_as_float(w.w), v[4 * i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w4 = q[i];
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = dtype == DG_BF16 ? BF16::unpack(w[j]) : F16::unpack(w[j]);
          v[8 * i + 2 * j] = fmaf(k, f.x, v[8 * i + 2 * j]);
          v[8 * i + 2 * j + 1] = fmaf(k, f.y, v[8 * i + 2 * j + 1]);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i] = fmaf(k, load_as_f32(p, i, dtype), v[i]);
  }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], "
      "[%1], %5;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z), "l"(policy_evict_first())
      : "memory");
}

// Where the 16-byte piece q of row r of a box lies: the swizzle of D's map,
// under which a warp's lanes, a row each, meet no bank conflicts.
__device__ __forceinline__ uint32_t box_offset(int r, int q) {
  return static_cast<uint32_t>(r * kBoxRow + ((q ^ (r & 7)) << 4));
}

// Sends a box (this warp's 32 rows, `pieces` of 16 bytes from column col0 on)
// to D (of the stack's matrix z): by TMA where all 32 rows are D's and the box
// is full or ends with D; else by the warp, eight lanes to a row of 16-byte
// pieces, or, where D's rows are not aligned so, all lanes to a row, 4 bytes
// each.  Either way lane 0 closes one bulk group.
//
// Params has D and its layout (D, N, ldd, stride_d, dtype_d, tma_d: TMA can
// store it, vec_d: its rows are 16-byte aligned), Tile its first row and rows.
template <typename Params, typename Tile>
__device__ __forceinline__ void send_box(const CUtensorMap* tmap_d, const uint8_t* box,
                                         const Params& p, const Tile& tile, int row_in_tile,
                                         int col0, int pieces, int matrix, int lane) {
  const int left = min(32, tile.rows - row_in_tile);  // rows of the box that are D's
  const int z = p.dtype_d == DG_F32 ? 4 : 2;
  const int per = 16 / z;  // columns in 16 bytes
  if (p.tma_d && left == 32 && (pieces == kBoxRow / 16 || col0 + pieces * per >= p.N)) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(tmap_d, box, col0, tile.row0 + row_in_tile, matrix);
      bulk_commit_group();
    }
    return;
  }
  if (lane == 0) bulk_commit_group();
  __syncwarp();
  const int64_t row = tile.row0 + row_in_tile;
  uint8_t* d = static_cast<uint8_t*>(p.D) + (matrix * p.stride_d + row * p.ldd + col0) * z;
  const int64_t pitch = p.ldd * z;
  const int bytes = min(pieces * 16, (p.N - col0) * z);  // of a row
  if (p.vec_d) {
    const int at = (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r >= left || at >= bytes) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(box + box_offset(r, lane & 7));
      uint8_t* dst = d + r * pitch + at;
      if (at + 16 <= bytes) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t h = w[k >> 1] >> (16 * (k & 1));
          if (at + 2 * k < bytes) reinterpret_cast<uint16_t*>(dst)[k] = static_cast<uint16_t>(h);
        }
      }
    }
    return;
  }
  const int at = lane * 4;
  if (at >= bytes) return;
  const bool whole = at + 4 <= bytes && (pitch & 3) == 0 && (p.stride_d * z & 3) == 0;
#pragma unroll 8
  for (int r = 0; r < left; ++r) {
    const uint32_t v =
        *reinterpret_cast<const uint32_t*>(box + box_offset(r, lane >> 2) + (lane & 3) * 4);
    uint8_t* dst = d + r * pitch + at;
    if (whole) {
      *reinterpret_cast<uint32_t*>(dst) = v;
    } else {
      reinterpret_cast<uint16_t*>(dst)[0] = static_cast<uint16_t>(v);
      if (at + 4 <= bytes) reinterpret_cast<uint16_t*>(dst)[1] = static_cast<uint16_t>(v >> 16);
    }
  }
}

// D as a stack of `count` matrices: boxes of 32 rows x 128 bytes, 128-byte
// swizzle.
inline cudaError_t make_out_map(CUtensorMap* map, const void* base, dg_dtype dtype, int64_t rows,
                         int64_t cols, int64_t ld, int64_t count, int64_t stride) {
  tc::EncodeTiledFn fn = tc::encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const int z = dtype == DG_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(count)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * z),
                                 static_cast<cuuint64_t>((count > 1 ? stride : rows * ld) * z)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBoxRow / z), 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == DG_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == DG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace fp8
}  // namespace dg
