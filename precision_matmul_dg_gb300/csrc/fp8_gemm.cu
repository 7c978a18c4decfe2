// FP8 (E4M3) products with FP32 block scales on tcgen05 (sm_103a): one dense
// product, one product per expert over rows sorted by expert, or one weight
// gradient per expert (dg_gemm_fp8, dg_gemm_fp8_grouped, ..._wgrad in dg.h).
//
//   t[i,j] = sum over 128-wide blocks b of K of  sa[i,b] * sb[j,b] * P_b[i,j],
//   P_b[i,j] = sum over k in b of A[i,k] * B[j,k]
//
// The tensor core adds within a block; scales change from block to block, so
// each block's P_b (one pipeline stage: 128 bytes of K) lands in a tensor
// memory buffer of its own and the epilogue warps add s * P_b to sums that
// stay in registers:
//
//   warps 0-7   sums and epilogue: warps w and w + 4 own TMEM lanes
//               32 * (w % 4) .. +31 (rows of D) and one half of the columns
//               each; per K block tcgen05.ld, then one packed FP32 FMA per two
//               columns with s = sa[i,b] * sb[b] (128 x 128 weight blocks: one
//               factor for the thread's row and half), or a multiplication by
//               the column's scale first (1 x 128 blocks in B);
//   warp 8      TMA producer of a ring of stages (A: 128 rows, B: BN rows, 128
//               bytes each, 128-byte swizzle);
//   warp 9      tensor memory allocation; MMA issuer, 4 x tcgen05.mma
//               (kind::f8f6f4, K = 32) per stage.
//
//   warp 10     with 1 x 128 blocks in B: brings the columns' scales of four K
//               blocks at a time to shared memory, two such groups ahead;
//   warp 11     nothing: it completes the third warpgroup.
//
// A sum thread holds 128 sums beside a 32-column load, more than the 168
// registers that 384 threads can have each: the third warpgroup keeps 72 and
// the two of the sum warps take 216 (2 x 216 + 72 = 3 x 168).
//
// The kernel is persistent: CTA u takes tiles u, u + grid, ...  Experts'
// segments are read from the device's offsets: every CTA counts the segments'
// 128-row blocks into shared memory, and every role walks the same tile list.
// A row tile may run into the next expert's rows (they are loaded, never
// stored).  Weight gradients walk (expert, tile) with K = the segment.
#include <algorithm>

#include "epilogue.cuh"
#include "fp8.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kTcThreads = 384;
constexpr int kLaunchRegs = 168, kSumRegs = 216, kOtherRegs = 72;  // per thread
static_assert(2 * kSumRegs + kOtherRegs == 3 * kLaunchRegs, "shares of the launch's registers");
constexpr int kColGroup = 4;  // K blocks whose column scales are staged together
constexpr int kSumWarps = 8;
constexpr int kRowsPerTile = 128;  // TMEM lanes
constexpr int kStageA = kRowsPerTile * 128;

struct F8Params {
  int M, N;  // kRows: M rows in all
  int m_blocks, n_blocks, k_blocks;
  int tiles;  // kDense, kK
  int group_m, count;
  int b_rows;  // rows of B's map from one expert to the next
  const int32_t* offsets;
  const float* sa;
  int64_t lds_a;
  const float* sb;
  int64_t lds_b, stride_sb;
  void* D;
  int64_t ldd, stride_d;
  const void* bias;
  int64_t stride_bias;
  float alpha, beta;
  int flags, dtype_d, vec;  // vec: bytes per store that D's layout allows (32, 16 or 0)
  uint32_t stage_tx;
  int k_rows;  // kK: rows of the sorted batch
  int* status;
  uint64_t timeout_ns;
};

template <int BN, int Stages, bool ColScale>
struct F8Smem {
  static constexpr int kTileB = BN * 128;
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + Stages * kStageA;
  static constexpr int kOffCol = kOffB + Stages * kTileB;  // column scales: [2][4][BN]
  static constexpr int kOffBar = kOffCol + (ColScale ? 2 * kColGroup * BN * 4 : 0);
  static constexpr int kBufs = 512 / BN < 4 ? 512 / BN : 4;
  static constexpr int kBars = 2 * Stages + 2 * kBufs + 1 + 4;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kOffGroups = (kOffAbort + 4 + 15) / 16 * 16;
  static constexpr int kFixed = kOffGroups + 1024;  // base alignment
  // row offsets and block counts of the experts, count + 1 each
  static int bytes(int64_t count) { return kFixed + static_cast<int>(2 * (count + 1) * 4); }
};

// One tile: rows row0 .. row0 + rows - 1 of A and D, columns from n0, K blocks
// [kb0, kb1).
struct F8Tile {
  int row0, rows, n0, expert, kb0, kb1;
};

struct F8Walk {
  int t, expert;
};

// The CTA's next tile; false past its last.  `off` and `pre` are the experts'
// row offsets and running 128-row block counts (kRows), off the K blocks (kK).
template <Fp8Mode Mode, int BN>
__device__ __forceinline__ bool next_tile(F8Walk& w, const F8Params& p, const int* off,
                                          const int* pre, F8Tile& o) {
  if (Mode == Fp8Mode::kRows) {
    while (w.expert < p.count && w.t >= pre[w.expert + 1] * p.n_blocks) ++w.expert;
    if (w.expert >= p.count) return false;
    const int mb = pre[w.expert + 1] - pre[w.expert];
    const int local = w.t - pre[w.expert] * p.n_blocks;
    const int nb = local / mb, m = local - nb * mb;  // rows first: concurrent tiles share weights
    o.expert = w.expert;
    o.row0 = off[w.expert] + m * kRowsPerTile;
    o.rows = min(kRowsPerTile, off[w.expert + 1] - o.row0);
    o.n0 = nb * BN;
    o.kb0 = 0;
    o.kb1 = p.k_blocks;
  } else {
    if (w.t >= p.tiles) return false;
    int local = w.t, m, nb;
    o.expert = 0;
    o.kb0 = 0;
    o.kb1 = p.k_blocks;
    if (Mode == Fp8Mode::kK) {
      const int per = p.m_blocks * p.n_blocks;
      o.expert = w.t / per;
      local = w.t - o.expert * per;
      o.kb0 = off[o.expert];
      o.kb1 = max(off[o.expert + 1], o.kb0);
    }
    tc::tile_coords(local, p.m_blocks, p.n_blocks, p.group_m, m, nb);
    o.row0 = m * kRowsPerTile;
    o.rows = min(kRowsPerTile, p.M - o.row0);
    o.n0 = nb * BN;
  }
  w.t += static_cast<int>(gridDim.x);
  return true;
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
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

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == DG_F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == DG_BF16 ? BF16::one(h) : F16::one(h);
}

// epilogue(alpha * t + beta * D) of 16 columns from col0 on, stored at D's row
// `drow` (element offset) for the columns < N.
__device__ __forceinline__ void finish16(float (&v)[16], const F8Params& p, int64_t drow, int col0,
                                         const void* bias, int64_t bias0) {
  const int n = p.N - col0;
  if (n <= 0) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= p.alpha;
  if (p.beta != 0.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i] = fmaf(p.beta, load_as_f32(p.D, drow + col0 + i, p.dtype_d), v[i]);
  }
  if (p.flags & kEpiBias) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i] += load_as_f32(bias, bias0 + col0 + i, p.dtype_d);
  }
  if (p.flags & kEpiGelu) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = gelu_erf(v[i]);
  }
  const bool full = n >= 16;
  if (p.dtype_d == DG_F32) {
    float* d = static_cast<float*>(p.D) + drow + col0;
    if (full && p.vec >= 16) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        reinterpret_cast<float4*>(d)[q] =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) d[i] = v[i];
    }
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    w[q] = p.dtype_d == DG_BF16 ? BF16::pack(v[2 * q], v[2 * q + 1])
                                : F16::pack(v[2 * q], v[2 * q + 1]);
  uint16_t* d = static_cast<uint16_t*>(p.D) + drow + col0;
  if (full && p.vec >= 16) {
    reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) d[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

template <Fp8Mode Mode, int BN, int Stages, bool ColScale>
__global__ void __launch_bounds__(kTcThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ F8Params p) {
  using L = F8Smem<BN, Stages, ColScale>;
  constexpr int kBufs = L::kBufs;
  constexpr int kHalf = BN / 2;  // columns per sum warp
  constexpr int kTmemCols = kBufs * BN;
  static_assert(kHalf % 32 == 0 && kTmemCols <= 512, "tile width");
  constexpr uint32_t idesc = idesc_f16_f32(kRowsPerTile, BN);  // operand format 0 is E4M3 here

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* col_scale = reinterpret_cast<float*>(smem + L::kOffCol);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty_bar = full_bar + Stages;
  uint64_t* tmem_full = empty_bar + Stages;
  uint64_t* tmem_empty = tmem_full + kBufs;
  uint64_t* drain_bar = tmem_empty + kBufs;
  uint64_t* col_full = drain_bar + 1;  // ColScale: the two groups of column scales
  uint64_t* col_empty = col_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  int* off = reinterpret_cast<int*>(smem + L::kOffGroups);
  int* pre = off + p.count + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], kSumWarps);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&col_full[g], 1);
      mbar_init(&col_empty[g], kSumWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
  }
  if (warp == 9) tmem_alloc<kTmemCols>(tmem_slot);
  // Launched as a programmatic dependent: everything above is this CTA's own
  // on-chip state; global memory waits for the kernel before.
  grid_dependency_wait();
  if (Mode != Fp8Mode::kDense) {
    // Offsets clamped to the rows there are (kK: in K blocks, rounded down).
    const int limit = Mode == Fp8Mode::kRows ? p.M : p.k_rows;
    bool odd = false;
    for (int e = threadIdx.x; e <= p.count; e += kTcThreads) {
      const int v = min(max(__ldg(p.offsets + e), 0), limit);
      odd |= Mode == Fp8Mode::kK && (v & (kBlock - 1)) != 0;
      off[e] = Mode == Fp8Mode::kK ? v / kBlock : v;
    }
    if (odd && blockIdx.x == 0) atomicExch(p.status, static_cast<int>(DG_ERR_INVALID_ARG));
    __syncthreads();
    if (Mode == Fp8Mode::kRows && warp == 0) {
      int run = 0;
      if (lane == 0) pre[0] = 0;
      for (int e0 = 0; e0 < p.count; e0 += 32) {
        const int e = e0 + lane;
        int v = 0;
        if (e < p.count)
          v = (max(off[e + 1] - off[e], 0) + kRowsPerTile - 1) / kRowsPerTile;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v += u;
        }
        if (e < p.count) pre[e + 1] = run + v;
        run += __shfl_sync(0xffffffffu, v, 31);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;
  F8Walk walk{static_cast<int>(blockIdx.x), 0};
  F8Tile tile;

  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ------------------------------------------------------------ producer
      if (elect_one_lane()) {
        const uint64_t pol = policy_evict_last();  // tiles are read again by other CTAs
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        while (ok && next_tile<Mode, BN>(walk, p, off, pre, tile)) {
          const int b_row = (Mode == Fp8Mode::kRows ? tile.expert * p.b_rows : 0) + tile.n0;
          for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
            if (!mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status,
                                     abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full_bar[stage], p.stage_tx);
            tma_load_2d(&tmap_a, &full_bar[stage], smem + L::kOffA + stage * kStageA, kb * kBlock,
                        tile.row0, pol);
            tma_load_2d(&tmap_b, &full_bar[stage], smem + L::kOffB + stage * L::kTileB, kb * kBlock,
                        b_row, pol);
            ++issued;
            if (++stage == Stages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        grid_launch_dependents();
        if (!ok) *abort_flag = 1;
        // the copies this thread started land before the CTA goes away, whoever gave up
        const int64_t first = issued > Stages ? issued - Stages : 0;
        for (int64_t i = first; i < issued; ++i)
          mbar_wait(&full_bar[i % Stages], static_cast<uint32_t>((i / Stages) & 1), p.timeout_ns,
                    p.status);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issuer
      if (elect_one_lane()) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        while (ok && next_tile<Mode, BN>(walk, p, off, pre, tile)) {
          for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
            if (!mbar_wait_abortable(&tmem_empty[buf], buf_phase ^ 1, p.timeout_ns, p.status,
                                     abort_flag) ||
                !mbar_wait_abortable(&full_bar[stage], phase, p.timeout_ns, p.status, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t da = smem_desc_sw128(smem_addr(smem + L::kOffA + stage * kStageA));
            const uint64_t db = smem_desc_sw128(smem_addr(smem + L::kOffB + stage * L::kTileB));
            // K step k starts 32 bytes further into the swizzled rows: +2 in the
            // descriptor's 16-byte address field
  #pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f8(tmem_base + static_cast<uint32_t>(buf * BN), da + 2 * k, db + 2 * k, idesc,
                        k != 0);
            tc_commit(&empty_bar[stage]);
            tc_commit(&tmem_full[buf]);
            if (++stage == Stages) {
              stage = 0;
              phase ^= 1;
            }
            if (++buf == kBufs) {
              buf = 0;
              buf_phase ^= 1;
            }
          }
        }
        if (!ok) *abort_flag = 1;
        tc_commit(drain_bar);  // the MMAs issued end before the tensor memory is freed
        mbar_wait(drain_bar, 0, p.timeout_ns, p.status);
      }
    } else if (ColScale && warp == 10) {
      // -------------------------------------------------------- column scales
      int g = 0;
      uint32_t g_phase = 0;
      while (ok && next_tile<Mode, BN>(walk, p, off, pre, tile)) {
        for (int kb = tile.kb0; kb < tile.kb1; kb += kColGroup) {
          ok = mbar_wait_abortable(&col_empty[g], g_phase ^ 1, p.timeout_ns, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float v[kColGroup][BN / 32];
#pragma unroll
          for (int i = 0; i < BN / 32; ++i) {
            const float* sb = p.sb + min(tile.n0 + lane + 32 * i, p.N - 1) * p.lds_b;
#pragma unroll
            for (int k = 0; k < kColGroup; ++k)
              v[k][i] = kb + k < tile.kb1 ? __ldg(sb + kb + k) : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < kColGroup; ++k)
#pragma unroll
            for (int i = 0; i < BN / 32; ++i)
              col_scale[(g * kColGroup + k) * BN + lane + 32 * i] = v[k][i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&col_full[g]);
          if (++g == 2) {
            g = 0;
            g_phase ^= 1;
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    // ------------------------------------------------------ sums and epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;
    int buf = 0, g = 0;
    uint32_t buf_phase = 0, g_phase = 0;
    while (ok && next_tile<Mode, BN>(walk, p, off, pre, tile)) {
      float2 acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      const int col0 = tile.n0 + half * kHalf;
      const float* sa = p.sa + static_cast<int64_t>(tile.row0 + min(r, tile.rows - 1)) * p.lds_a;
      const float* sb = p.sb + (Mode == Fp8Mode::kRows ? tile.expert * p.stride_sb : 0) +
                        static_cast<int64_t>(min(col0, p.N - 1) / kBlock) * p.lds_b;
      float a_next = 0.0f, b_next = 1.0f;
      if (tile.kb0 < tile.kb1) {
        a_next = __ldg(sa + tile.kb0);
        if (!ColScale) b_next = __ldg(sb + tile.kb0);
      }
      for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
        const float s = a_next * b_next;
        if (kb + 1 < tile.kb1) {
          a_next = __ldg(sa + kb + 1);
          if (!ColScale) b_next = __ldg(sb + kb + 1);
        }
        const int in_group = (kb - tile.kb0) % kColGroup;
        if (ColScale && in_group == 0)
          ok = mbar_wait_abortable(&col_full[g], g_phase, p.timeout_ns, p.status, abort_flag);
        ok = ok && mbar_wait_abortable(&tmem_full[buf], buf_phase, p.timeout_ns, p.status,
                                       abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const float2 s2 = make_float2(s, s);
        const uint32_t src = tmem_base + lane_base + static_cast<uint32_t>(buf * BN + half * kHalf);
        const float* cs = col_scale + (g * kColGroup + in_group) * BN + half * kHalf;
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t v[32];
          tmem_ld_32cols(src + c, v);
          tc_wait_ld();
          if (c + 32 >= kHalf) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tmem_empty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 x = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            if (ColScale) x = mul2(x, *reinterpret_cast<const float2*>(cs + c + 2 * i));
            acc[c / 2 + i] = fma2(x, s2, acc[c / 2 + i]);
          }
        }
        if (++buf == kBufs) {
          buf = 0;
          buf_phase ^= 1;
        }
        if (ColScale && (in_group == kColGroup - 1 || kb + 1 == tile.kb1)) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&col_empty[g]);
          if (++g == 2) {
            g = 0;
            g_phase ^= 1;
          }
        }
      }
      if (!ok) break;
      if (r < tile.rows) {
        const int64_t drow = (Mode == Fp8Mode::kK ? tile.expert * p.stride_d : 0) +
                             static_cast<int64_t>(tile.row0 + r) * p.ldd;
        const int64_t bias0 = Mode == Fp8Mode::kRows ? tile.expert * p.stride_bias : 0;
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = acc[c / 2 + i].x;
            v[2 * i + 1] = acc[c / 2 + i].y;
          }
          finish16(v, p, drow, col0 + c, p.bias, bias0);
        }
      }
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc<kTmemCols>(tmem_base);
  }
}

template <Fp8Mode Mode, int BN, int Stages, bool ColScale>
cudaError_t run_fp8(const Fp8Args& a) {
  using L = F8Smem<BN, Stages, ColScale>;
  const int box_a = Mode == Fp8Mode::kDense && a.M < kRowsPerTile
                        ? static_cast<int>((a.M + 7) / 8 * 8)
                        : kRowsPerTile;
  CUtensorMap ta, tb;
  cudaError_t e = tc::make_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, a.M, a.K, a.lda, box_a,
                                  128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int64_t b_pitch = Mode == Fp8Mode::kRows ? a.stride_b / a.ldb : 0;
  const int64_t b_rows = Mode == Fp8Mode::kRows ? (a.count - 1) * b_pitch + a.N : a.N;
  e = tc::make_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, b_rows, a.K, a.ldb, BN, 128,
                      CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  F8Params p;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.m_blocks = static_cast<int>((a.M + kRowsPerTile - 1) / kRowsPerTile);
  p.n_blocks = static_cast<int>((a.N + BN - 1) / BN);
  p.k_blocks = static_cast<int>((a.K + kBlock - 1) / kBlock);
  p.k_rows = static_cast<int>(a.K);
  const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_blocks *
                        (Mode == Fp8Mode::kK ? a.count : 1);
  p.tiles = static_cast<int>(std::min<int64_t>(tiles, INT32_MAX));
  p.group_m = 16;
  p.count = Mode == Fp8Mode::kDense ? 0 : static_cast<int>(a.count);
  p.b_rows = static_cast<int>(b_pitch);
  p.offsets = a.offsets;
  p.sa = a.sa;
  p.lds_a = a.lds_a;
  p.sb = a.sb;
  p.lds_b = a.lds_b;
  p.stride_sb = a.stride_sb;
  p.D = a.D;
  p.ldd = a.ldd;
  p.stride_d = a.stride_d;
  p.bias = a.bias;
  p.stride_bias = a.stride_bias;
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.flags = a.epi;
  p.dtype_d = static_cast<int>(a.dtype_d);
  const int64_t z = a.dtype_d == DG_F32 ? 4 : 2;
  p.vec = (a.ldd * z) % 16 == 0 && (a.stride_d * z) % 16 == 0 ? 16 : 0;
  p.stage_tx = static_cast<uint32_t>(box_a * 128 + L::kTileB);
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;

  auto kern = gemm_fp8_kernel<Mode, BN, Stages, ColScale>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  e = once_per_device(attr_set, dev, [&]() {
    // the warpgroups' shares of the registers hold for this count only: with
    // fewer at launch, the sum warps would wait for registers without end
    cudaFuncAttributes fa{};
    const cudaError_t r = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kern));
    if (r != cudaSuccess) return r;
    if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::bytes(Mode == Fp8Mode::kDense ? 0 : kMaxExperts));
  });
  if (e != cudaSuccess) return e;
  // Experts' tiles are counted on the device: at most one part-filled row
  // block per expert beside the full ones.
  const int64_t most = Mode == Fp8Mode::kRows
                           ? (a.M / kRowsPerTile + std::min(a.count, a.M)) * p.n_blocks
                           : tiles;
  if (most > (1 << 30)) return cudaErrorInvalidConfiguration;  // tile numbers are 32-bit
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(most, a.sm_count));
  e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kTcThreads),
                       static_cast<size_t>(L::bytes(p.count)), a.stream, ta, tb, p);
  count_launches(1);
  return e;
}

template <Fp8Mode Mode>
cudaError_t run_mode(const Fp8Args& a) {
  if (a.block_rows_b == 1) return run_fp8<Mode, 256, 4, true>(a);
  return run_fp8<Mode, 256, 4, false>(a);
}

}  // namespace

cudaError_t launch_fp8_tc(const Fp8Args& a) {
  switch (a.mode) {
    case Fp8Mode::kDense: return run_mode<Fp8Mode::kDense>(a);
    case Fp8Mode::kRows: return run_fp8<Fp8Mode::kRows, 256, 4, false>(a);
    case Fp8Mode::kK: return run_fp8<Fp8Mode::kK, 256, 4, true>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dg
