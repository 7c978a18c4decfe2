// Block quantization of FP16 / BF16 rows to E4M3 codes with FP32 scales
// (dg_quantize_fp8), and the same on rows gathered by expert
// (dg_moe_dispatch_fp8).
//
// For a block with largest magnitude amax (at least 448 * 2^-126):
//   scale = amax / 448,  code = e4m3(v * (448 / amax)),
// both quotients and the product rounded to FP32, the code to nearest even.
// The magnitudes are compared as 16-bit patterns (sign cleared), which orders
// finite values and puts infinities and NaNs above them; such a block gets
// codes 0 and the scale NaN.
//
// Bound by memory: 2 bytes read and 1 written per value (2 written with both
// forms), so the row kernel keeps a row's loads contiguous and several rows
// in flight per thread, and the tile kernel makes the row form and the
// transposed form out of one read of a 128 x 128 tile.
#include <cuda_runtime.h>

#include "fp8.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 ld_nc16(const void* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// 16 consecutive values of a row as 8 words; zeros past n values.
__device__ __forceinline__ void load16(const uint16_t* p, int64_t n, uint32_t (&w)[8]) {
  if (n >= 16) {
    const uint4 a = ld_nc16(p), b = ld_nc16(p + 8);
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

// Codes of 16 values, stored at dst for the first n of them.
template <typename T>
__device__ __forceinline__ void store_codes16(const uint32_t (&w)[8], const BlockScale& b,
                                              uint8_t* dst, int64_t n) {
  const uint32_t lo[4] = {w[0], w[1], w[2], w[3]}, hi[4] = {w[4], w[5], w[6], w[7]};
  const uint2 c0 = quantize8<T>(lo, b), c1 = quantize8<T>(hi, b);
  if (n >= 16) {
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(c0.x, c0.y, c1.x, c1.y));
  } else {
    const uint32_t c[4] = {c0.x, c0.y, c1.x, c1.y};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) dst[i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
  }
}

// Row form, 1 x 128 blocks.  Eight lanes take a block, 16 values (32 bytes)
// each; 2^log2_tpr threads share a row, and each thread has kRows rows in
// flight (8192 x 4096: 15.2 us, 6640 GB/s; 16 x 4096 1.8 us).  With a gather
// (row_slot), row r is X's row row_slot[r] / top_k, or zeros when the slot is -1
// or past the tokens.
constexpr int kRows = 2;

struct RowParams {
  const uint16_t* X;
  int64_t ldx, rows, K;
  int nblk, log2_tpr;
  uint8_t* codes;
  int64_t ldq;
  float* scales;
  int64_t lds;
  const int32_t* row_slot;  // NULL: no gather
  int top_k;
  int64_t tokens;
};

template <typename T, bool Gather>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const __grid_constant__ RowParams p) {
  grid_dependency_wait();  // launched as a dependent of the previous kernel
  grid_launch_dependents();
  const int tpr = 1 << p.log2_tpr;
  const int in_row = threadIdx.x & (tpr - 1);
  const int rows_per_pass = kThreads >> p.log2_tpr;
  const int sub = in_row & 7;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_pass;
  // bounds are the same for all lanes of a warp: every lane takes part in the
  // shuffles
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_per_pass; base < p.rows;
       base += step * kRows) {
    const uint16_t* src[kRows];
    int64_t row[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      row[i] = base + i * step + (threadIdx.x >> p.log2_tpr);
      src[i] = nullptr;
      if (row[i] < p.rows) {
        if (Gather) {
          const int slot = __ldg(p.row_slot + row[i]);
          const int t = slot < 0 ? -1 : static_cast<int>(static_cast<unsigned>(slot) / p.top_k);
          if (t >= 0 && t < p.tokens) src[i] = p.X + t * p.ldx;
        } else {
          src[i] = p.X + row[i] * p.ldx;
        }
      }
    }
    for (int b0 = 0; b0 < p.nblk; b0 += tpr >> 3) {
      const int b = b0 + (in_row >> 3);
      const int64_t k = static_cast<int64_t>(b) * kBlock + sub * 16;
      const int64_t n = b < p.nblk ? p.K - k : 0;
      uint32_t w[kRows][8];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[i][q] = 0u;
        if (src[i] && n > 0) load16(src[i] + k, n, w[i]);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        uint32_t m = amax_bits16(w[i]);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (row[i] >= p.rows || b >= p.nblk) continue;
        const BlockScale s = block_scale<T>(m);
        if (n > 0) store_codes16<T>(w[i], s, p.codes + row[i] * p.ldq + k, n);
        if (sub == 0) p.scales[row[i] * p.lds + b] = s.scale;
      }
    }
  }
}

// A 128 x 128 tile: row form and / or transposed form, with 1 x 128 blocks
// (of the respective form's rows) or one block for the whole tile.  Thread t
// reads 16 values of rows t / 8 + 32 i, makes their row-form codes, and puts
// them in shared memory; then it takes two columns and a quarter of the rows
// for the transposed form, whose codes go back through shared memory and out
// as whole 128-byte lines.  (8192 x 4096, both forms: 29.1 us, 4610 GB/s, one
// scale per tile 25.8; transposed alone 20.0 us, 5030 GB/s; 8191 rows, whose
// transposed rows of codes are not aligned, 31.3.  Bound by the phases of a tile
// more than by memory: instructions issue in 49% of the clocks.)
constexpr int kPitch = kBlock + 8;       // 16-bit elements per shared row
constexpr int kCodePitch = kBlock + 16;  // bytes per shared column of codes
static_assert(kBlock * kCodePitch <= kBlock * kPitch * 2, "the codes take the tile's place");

struct TileParams {
  const uint16_t* X;
  int64_t ldx, rows, K;
  int col_tiles;
  int whole;  // one block per tile (block_rows 128)
  uint8_t* codes;
  int64_t ldq;
  float* scales;
  int64_t lds;
  uint8_t* codes_t;
  int64_t ldqt;
  float* scales_t;
  int64_t ldst;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_tile_kernel(const __grid_constant__ TileParams p) {
  __shared__ __align__(16) uint16_t tile[kBlock * kPitch];
  __shared__ uint32_t col_max[4][kBlock / 2];
  __shared__ uint32_t warp_max[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const int64_t rt = blockIdx.x / p.col_tiles;
  const int ct = static_cast<int>(blockIdx.x - rt * p.col_tiles);
  const int64_t r0 = rt * kBlock, c0 = static_cast<int64_t>(ct) * kBlock;
  const int sub = t & 7;
  const int64_t n = p.K - (c0 + sub * 16);  // values of the row from this thread's first on

  uint32_t w[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + (t >> 3) + 32 * i;
#pragma unroll
    for (int q = 0; q < 8; ++q) w[i][q] = 0u;
    if (r < p.rows && n > 0) load16(p.X + r * p.ldx + c0 + sub * 16, n, w[i]);
  }
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = amax_bits16(w[i]);
  uint32_t whole_max = 0;
  if (p.whole) {
    whole_max = max(max(m[0], m[1]), max(m[2], m[3]));
    whole_max = __reduce_max_sync(0xffffffffu, whole_max);
    if ((t & 31) == 0) warp_max[t >> 5] = whole_max;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) whole_max = max(whole_max, warp_max[i]);
  }
  if (p.codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t mm = whole_max;
      if (!p.whole) {
        mm = m[i];
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) mm = max(mm, __shfl_xor_sync(0xffffffffu, mm, d));
      }
      const BlockScale s = block_scale<T>(mm);
      const int64_t r = r0 + (t >> 3) + 32 * i;
      if (r < p.rows) {
        if (n > 0) store_codes16<T>(w[i], s, p.codes + r * p.ldq + c0 + sub * 16, n);
        if (!p.whole && sub == 0) p.scales[r * p.lds + ct] = s.scale;
      }
      if (p.whole && i == 0 && t == 0) p.scales[rt * p.lds + ct] = s.scale;
    }
  }
  if (!p.codes_t) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4* d = reinterpret_cast<uint4*>(tile + ((t >> 3) + 32 * i) * kPitch + sub * 16);
    d[0] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    d[1] = make_uint4(w[i][4], w[i][5], w[i][6], w[i][7]);
  }
  __syncthreads();
  const int pair = t & 63, part = t >> 6;
  const uint32_t* col = reinterpret_cast<const uint32_t*>(tile) + part * 32 * (kPitch / 2) + pair;
  uint32_t lo_max = whole_max, hi_max = whole_max;
  if (!p.whole) {
    uint32_t cm = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) cm = __vmaxu2(cm, col[i * (kPitch / 2)] & 0x7FFF7FFFu);
    col_max[part][pair] = cm;
    __syncthreads();
    cm = __vmaxu2(__vmaxu2(col_max[0][pair], col_max[1][pair]),
                  __vmaxu2(col_max[2][pair], col_max[3][pair]));
    lo_max = cm & 0xFFFFu;
    hi_max = cm >> 16;
  }
  const BlockScale s[2] = {block_scale<T>(lo_max), block_scale<T>(hi_max)};
  uint32_t o[2][8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = T::unpack(col[(4 * q + i) * (kPitch / 2)]);
    const float f0 = s[0].factor, f1 = s[1].factor;
    o[0][q] = s[0].bad ? 0u : e4m3x4(v[0].x * f0, v[1].x * f0, v[2].x * f0, v[3].x * f0);
    o[1][q] = s[1].bad ? 0u : e4m3x4(v[0].y * f1, v[1].y * f1, v[2].y * f1, v[3].y * f1);
  }
  // through shared memory, so that eight lanes write a column's 128 bytes
  __syncthreads();  // the tile has been read
  uint8_t* ct_smem = reinterpret_cast<uint8_t*>(tile);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = 2 * pair + h;
    uint4* d = reinterpret_cast<uint4*>(ct_smem + c * kCodePitch + part * 32);
    d[0] = make_uint4(o[h][0], o[h][1], o[h][2], o[h][3]);
    d[1] = make_uint4(o[h][4], o[h][5], o[h][6], o[h][7]);
    if (!p.whole && part == 0 && c0 + c < p.K) p.scales_t[(c0 + c) * p.ldst + rt] = s[h].scale;
  }
  __syncthreads();
  const int64_t rr = r0 + sub * 16;  // a position along the output's rows
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (t >> 3) + 32 * i;
    if (c0 + c >= p.K || rr >= p.rows) break;
    const uint4 v = *reinterpret_cast<const uint4*>(ct_smem + c * kCodePitch + sub * 16);
    uint8_t* dst = p.codes_t + (c0 + c) * p.ldqt + rr;
    if (rr + 16 <= p.rows) {
      __stcs(reinterpret_cast<uint4*>(dst), v);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (rr + k < p.rows) dst[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
    }
  }
  if (p.whole && t == 0) p.scales_t[ct * p.ldst + rt] = s[0].scale;
}

template <typename T>
cudaError_t rows_launch(const RowParams& p, bool gather, dim3 grid, cudaStream_t stream) {
  auto kern = gather ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>;
  return launch_dependent(kern, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_quantize_fp8_rows(const Fp8RowsJob& j, cudaStream_t stream, int sm_count) {
  RowParams p;
  p.X = static_cast<const uint16_t*>(j.X);
  p.ldx = j.ldx;
  p.rows = j.rows;
  p.K = j.K;
  p.nblk = static_cast<int>((j.K + kBlock - 1) / kBlock);
  p.log2_tpr = 3;
  while (p.log2_tpr < 8 && (1 << p.log2_tpr) < p.nblk * 8) ++p.log2_tpr;
  p.codes = static_cast<uint8_t*>(j.codes);
  p.ldq = j.ldq;
  p.scales = j.scales;
  p.lds = j.lds;
  p.row_slot = j.row_slot;
  p.top_k = static_cast<int>(j.top_k);
  p.tokens = j.tokens;
  const int64_t per_cta = kThreads >> p.log2_tpr;
  const int64_t ctas = (j.rows + per_cta - 1) / per_cta;
  const int64_t cap = static_cast<int64_t>(sm_count) * 16;
  const dim3 grid(static_cast<unsigned>(ctas < cap ? ctas : cap));
  const bool gather = j.row_slot != nullptr;
  const cudaError_t e = j.bf16 ? rows_launch<BF16>(p, gather, grid, stream)
                               : rows_launch<F16>(p, gather, grid, stream);
  count_launches(1);
  return e;
}

cudaError_t launch_quantize_fp8_tiles(const Fp8TilesJob& j, cudaStream_t stream) {
  TileParams p;
  p.X = static_cast<const uint16_t*>(j.X);
  p.ldx = j.ldx;
  p.rows = j.rows;
  p.K = j.K;
  p.col_tiles = static_cast<int>((j.K + kBlock - 1) / kBlock);
  p.whole = j.whole ? 1 : 0;
  p.codes = static_cast<uint8_t*>(j.codes);
  p.ldq = j.ldq;
  p.scales = j.scales;
  p.lds = j.lds;
  p.codes_t = static_cast<uint8_t*>(j.codes_t);
  p.ldqt = j.ldqt;
  p.scales_t = j.scales_t;
  p.ldst = j.ldst;
  const int64_t tiles = (j.rows + kBlock - 1) / kBlock * p.col_tiles;
  const dim3 grid(static_cast<unsigned>(tiles));
  const cudaError_t e =
      j.bf16 ? launch_dependent(quantize_tile_kernel<BF16>, grid, dim3(kThreads), 0, stream, p)
             : launch_dependent(quantize_tile_kernel<F16>, grid, dim3(kThreads), 0, stream, p);
  count_launches(1);
  return e;
}

}  // namespace dg
