// FP8 (E4M3) products with FP32 block scales on tcgen05 (sm_103a): one dense
// product, one product per expert over rows sorted by expert, or one weight
// gradient per expert (dg_gemm_fp8, dg_gemm_fp8_grouped, ..._wgrad in dg.h).
//
//   t[i,j] = sum over 128-wide blocks b of K of  sa[i,b] * sb[j,b] * P_b[i,j],
//   P_b[i,j] = sum over k in b of A[i,k] * B[j,k]
//
// The tensor core adds within a block; scales change from block to block, so
// each block's P_b (one pipeline stage: 128 bytes of K) lands in a tensor
// memory buffer of its own and the sum warps add s * P_b to sums that stay in
// registers:
//
//   warps 0-7   sums and epilogue: warps w and w + 4 own TMEM lanes
//               32 * (w % 4) .. +31 (rows of D) and one half of the columns
//               each; per K block tcgen05.ld, then one packed FP32 FMA per two
//               columns with s = sa[i,b] * sb[b] (128 x 128 weight blocks: one
//               factor for the thread's row and half), or a multiplication by
//               the column's scale first (1 x 128 blocks in B);
//   warp 8      TMA producer of a ring of stages (128 rows of A, BN rows of B,
//               128 bytes each, 128-byte swizzle);
//   warp 9      tensor memory allocation; MMA issuer, 4 x tcgen05.mma
//               (kind::f8f6f4, K = 32) per stage;
//   warps 10-11 bring the scales of four K blocks at a time to shared memory,
//               two such groups ahead (a sum thread that loads its row's scale
//               itself reads 32 lines with 31 others; that cost 137 clocks a K
//               block): the rows' by TMA, the columns' (1 x 128 blocks in B)
//               transposed, half of them each, or the halves' weight blocks'.
//
// What a K block of a 128 x 256 tile takes is about 830 clocks, where its MMAs
// take 512 and its TMEM loads 560.  What fills the rest is not settled: an MMA
// waits for the release of the buffer before last, a release for the loads of
// the last column, and both for an mbarrier's way there; but the 128 x 128 tile
// with four buffers takes 0.6 of these clocks, with half the MMAs (8192^3: 458 us
// a call, 62% of the tensor rate, 425 in graph replays; 32768 x 4096 x 2048: 236
// us, 64 experts' 32768 rows of the same sizes, whose last tiles are part-filled:
// 287 us, with GELU 335; FP32 gradients of 64 experts, 4096 x 2048 each: 527 us,
// 4.07 TB/s of stores, what clearing such a buffer reaches; BF16 gradients 429
// us).  Measured with no gain: pairs of CTAs (cta_group::2, half of B
// each), two CTAs per SM with 128 x 128 tiles, a fourth stage, loads of 32
// columns.
//
// A sum thread holds up to 128 sums beside two 16-column loads, more than the
// 168 registers that 384 threads can have each: the third warpgroup keeps 72
// and the two of the sum warps take 216 (2 x 216 + 72 = 3 x 168).
//
// The kernel is persistent: CTA u takes tiles u, u + CTAs, ...  Experts'
// segments are read from the device's offsets: every CTA counts the segments'
// row blocks into shared memory, and every role walks the same tile list.  A
// row tile may run into the next expert's rows (they are loaded, never stored).
// Weight gradients walk (expert, tile) with K = the segment.  Split: a dense
// product of few tiles has a cluster of CTAs per tile, a share of K each, whose
// sums meet through distributed shared memory in the order of K.
//
// D leaves through shared memory: a warp's 32 rows x 128 bytes at a time,
// by TMA, or (a segment's last rows, layouts that TMA does not take) by the
// warp in runs of whole rows.  Straight from registers a store touches 32 rows, one
// line each: 5500 clocks per 128 x 256 tile.
#include <algorithm>
#include <type_traits>

#include "epilogue.cuh"
#include "fp8.cuh"
#include "out_box.cuh"
#include "segments.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kSumRegs = 216, kOtherRegs = 72;  // per thread
static_assert(2 * kSumRegs + kOtherRegs == 3 * kLaunchRegs, "shares of the launch's registers");
constexpr int kScaleGroup = 4;  // K blocks (of one number / 4) whose scales are staged together
constexpr int kSumWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kScaleWarp = 10;
constexpr int kRowsPerCta = 128;  // TMEM lanes
constexpr int kStageA = kRowsPerCta * 128;
constexpr int kRowScaleBytes = kRowsPerCta * kScaleGroup * 4;

struct F8Params {
  int M, N;  // kRows: M rows in all
  int m_blocks, n_blocks, k_blocks;
  int split, split_blocks;  // Split: CTAs per tile, and K blocks of each (whole scale groups)
  int tiles;  // kDense, kK
  int group_m, count;
  int b_rows;  // rows of B's map from one expert to the next
  const int32_t* offsets;
  uint32_t most_blocks;  // experts: row blocks whose tiles a walk takes
  const float* sa;
  int64_t lds_a;
  const float* sb;
  int64_t lds_b, stride_sb;
  void* D;
  int64_t ldd, stride_d;
  const void* bias;
  int64_t stride_bias;
  float alpha, beta;
  int flags, dtype_d;
  int tma_d, vec_d;  // D's layout: TMA can store it; rows are 16-byte aligned
  int vec_a, vec_b;  // rows of scales are too
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
  static constexpr int kOffBox = kOffB + Stages * kTileB;
  static constexpr int kBoxes = BN == 256 ? 2 : 1;  // D's, per sum warp
  static constexpr int kOffRow = kOffBox + kSumWarps * kBoxes * kBoxBytes;  // [2][128][4]
  static constexpr int kOffCol = kOffRow + 2 * kRowScaleBytes;
  // column scales [2][4][BN], or the halves' block scales [2][2][4]
  static constexpr int kOffBar = kOffCol + 2 * kScaleGroup * (ColScale ? BN : 2) * 4;
  static constexpr int kBufs = 512 / BN;
  static constexpr int kBars = 2 * Stages + 2 * kBufs + 1 + 4;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kOffGroups = (kOffAbort + 4 + 15) / 16 * 16;
  static constexpr int kFixed = kOffGroups + 1024;  // base alignment
  // count + 1 row offsets of the experts, and without column scales (kRows) as
  // many row block counts
  static constexpr int bytes(int64_t count) {
    return kFixed + static_cast<int>(count > 0 ? (ColScale ? 1 : 2) * (count + 1) * 4 : 0);
  }
  static_assert(bytes(kMaxExperts) <= 227 * 1024, "shared memory of a CTA");
};

// A tile: rows row0 .. row0 + rows - 1 of A and D, columns from n0, K blocks
// [kb0, kb1).
struct F8Tile {
  int row0, rows, n0, expert, kb0, kb1;
};

struct F8Walk {
  int t, expert, rank;  // rank: the CTA's share of K (Split)
};

// The CTA's next tile; false past its last.  `off` and `pre` are the experts'
// row offsets and running row block counts (kRows), off the K blocks (kK).
template <Fp8Mode Mode, int BN, bool Split>
__device__ __forceinline__ bool next_tile(F8Walk& w, const F8Params& p, const int* off,
                                          const int* pre, F8Tile& o) {
  if (Mode == Fp8Mode::kRows) {
    while (w.expert < p.count && w.t >= pre[w.expert + 1] * p.n_blocks) ++w.expert;
    if (w.expert >= p.count) return false;
    const int mb = pre[w.expert + 1] - pre[w.expert];
    const int local = w.t - pre[w.expert] * p.n_blocks;
    const int nb = local / mb, m = local - nb * mb;  // rows first: concurrent tiles share weights
    o.expert = w.expert;
    o.row0 = off[w.expert] + m * kRowsPerCta;
    o.rows = min(kRowsPerCta, off[w.expert + 1] - o.row0);
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
    if (Split) {
      o.kb0 = min(w.rank * p.split_blocks, p.k_blocks);
      o.kb1 = min(o.kb0 + p.split_blocks, p.k_blocks);
    }
    tc::tile_coords(local, p.m_blocks, p.n_blocks, p.group_m, m, nb);
    o.row0 = m * kRowsPerCta;
    o.rows = min(kRowsPerCta, p.M - o.row0);
    o.n0 = nb * BN;
  }
  w.t += Split ? p.tiles : static_cast<int>(gridDim.x);  // a split tile is the CTA's only one
  return true;
}

// One K block: four MMAs (K = 32 each, 32 bytes further into the swizzled rows:
// +2 in the descriptors' 16-byte address field) into d_tmem, whose end arrives
// on done_bar (the buffer is full) and free_bar (the stage is free).  Issued by
// the lane with `issue` set, without a branch.
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t done_bar, uint32_t free_bar,
                                          uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred i, f, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.u32 i, %6, 0;\n\t"
      "setp.ne.u32 f, 0, 0;\n\t"
      "setp.eq.u32 t, 0, 0;\n\t"
      "@i tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
      "add.s64 a, %1, 2;\n\t"
      "add.s64 b, %2, 2;\n\t"
      "@i tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\t"
      "add.s64 b, %2, 4;\n\t"
      "@i tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\t"
      "add.s64 b, %2, 6;\n\t"
      "@i tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "@i tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
      "@i tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
      :
      : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(done_bar), "r"(free_bar), "r"(issue)
      : "memory");
}

// A wait of a whole warp, all lanes polling together so that the warp stays
// converged: one lane polling for the others costs 240 clocks a time, this 50.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const F8Params& p,
                                          volatile int* abort) {
  const uint32_t a = smem_addr(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > p.timeout_ns)) {
      atomicExch(p.status, kStatusTimeout);
      return false;
    }
  }
}

// tcgen05.wait::ld that names the registers it makes readable, so that no use
// of them is moved above it.
__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The scales of K blocks kb .. kb + 3 (kb a multiple of 4, vec: rows of scales
// are 16-byte aligned) of a row of nk; past its end, whatever is read instead
// is not used.  Nothing is done with the values here: a select after the load
// would wait for it.
__device__ __forceinline__ void load_group(float4& v, const float* s, int kb, int nk, int vec) {
  if (vec) {
    v = __ldg(reinterpret_cast<const float4*>(s + min(kb, (nk - 1) & ~(kScaleGroup - 1))));
  } else {
    v.x = __ldg(s + min(kb, nk - 1));
    v.y = __ldg(s + min(kb + 1, nk - 1));
    v.z = __ldg(s + min(kb + 2, nk - 1));
    v.w = __ldg(s + min(kb + 3, nk - 1));
  }
}

// alpha * t + beta * D, bias and GELU of 16 columns from col0 on, row `drow`
// (element offset of D).  Columns >= N read nothing.  Gradients have neither
// bias nor GELU.
template <Fp8Mode Mode>
__device__ __forceinline__ void finish16(float (&v)[16], const F8Params& p, int64_t drow, int col0,
                                         int64_t bias0) {
  const int n = p.N - col0;
  const int64_t z = p.dtype_d == DG_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= p.alpha;
  if (p.beta != 0.0f)
    add16(v, p.beta, static_cast<const uint8_t*>(p.D) + (drow + col0) * z, p.dtype_d, n);
  if (Mode != Fp8Mode::kK && (p.flags & kEpiBias))
    add16(v, 1.0f, static_cast<const uint8_t*>(p.bias) + (bias0 + col0) * z, p.dtype_d, n);
  if (Mode != Fp8Mode::kK && (p.flags & kEpiGelu)) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 g = gelu2(make_float2(v[i], v[i + 1]));
      v[i] = g.x;
      v[i + 1] = g.y;
    }
  }
}

__device__ __forceinline__ float4 ld_cluster_float4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <Fp8Mode Mode, int BN, int Stages, bool ColScale, bool Split>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_d,
                    const __grid_constant__ CUtensorMap tmap_sa,
                    const __grid_constant__ F8Params p) {
  using L = F8Smem<BN, Stages, ColScale>;
  constexpr int kBufs = L::kBufs;
  constexpr int kHalf = BN / 2;  // columns per sum warp
  constexpr int kTmemCols = kBufs * BN;
  constexpr uint32_t idesc = idesc_f16_f32(kRowsPerCta, BN);  // operand format 0 is E4M3 here

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* col_scale = reinterpret_cast<float*>(smem + L::kOffCol);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty_bar = full_bar + Stages;
  uint64_t* tmem_full = empty_bar + Stages;
  uint64_t* tmem_empty = tmem_full + kBufs;
  uint64_t* drain_bar = tmem_empty + kBufs;
  uint64_t* scale_full = drain_bar + 1;
  uint64_t* scale_empty = scale_full + 2;
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
      mbar_init(&scale_full[g], ColScale ? 2 : 1);
      mbar_init(&scale_empty[g], kSumWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
    tma_prefetch_desc(&tmap_d);
    tma_prefetch_desc(&tmap_sa);
  }
  if (warp == kMmaWarp) tmem_alloc<kTmemCols>(tmem_slot);
  // Launched as a programmatic dependent: everything above is this CTA's own
  // on-chip state; global memory waits for the kernel before.
  grid_dependency_wait();
  if (Mode != Fp8Mode::kDense) {
    // Offsets clamped to the rows there are (kK: in K blocks, rounded down).
    const int limit = Mode == Fp8Mode::kRows ? p.M : p.k_rows;
    bool odd = false;
    for (int e = threadIdx.x; e <= p.count; e += kThreads) {
      const int v = min(max(__ldg(p.offsets + e), 0), limit);
      odd |= Mode == Fp8Mode::kK && (v & (kBlock - 1)) != 0;
      off[e] = Mode == Fp8Mode::kK ? v / kBlock : v;
    }
    if (odd && blockIdx.x == 0) atomicExch(p.status, static_cast<int>(DG_ERR_INVALID_ARG));
    __syncthreads();
    if (Mode == Fp8Mode::kRows && warp == 0)
      count_row_blocks(off, pre, p.count, kRowsPerCta, p.most_blocks, blockIdx.x == 0, p.status, lane);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true, met = false;  // met: the cluster's first barrier (Split)
  F8Walk walk{static_cast<int>(blockIdx.x), 0, 0};
  if (Split) {
    walk.rank = static_cast<int>(cluster_ctarank());
    walk.t = static_cast<int>(blockIdx.x) / p.split;
  }
  F8Tile tile;

  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------- producer
      if (elect_one_lane()) {
        const uint64_t pol = policy_evict_last();  // tiles are read again by other CTAs
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        while (ok && next_tile<Mode, BN, Split>(walk, p, off, pre, tile)) {
          const int b_row = (Mode == Fp8Mode::kRows ? tile.expert * p.b_rows : 0) + tile.n0;
          for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
            if (!mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status,
                                     abort_flag)) {
              ok = false;
              break;
            }
            uint8_t* dst_a = smem + L::kOffA + stage * kStageA;
            uint8_t* dst_b = smem + L::kOffB + stage * L::kTileB;
            mbar_arrive_expect_tx(&full_bar[stage], p.stage_tx);
            tma_load_2d(&tmap_a, &full_bar[stage], dst_a, kb * kBlock, tile.row0, pol);
            tma_load_2d(&tmap_b, &full_bar[stage], dst_b, kb * kBlock, b_row, pol);
            ++issued;
            if (++stage == Stages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        grid_launch_dependents();
        if (!ok) *abort_flag = 1;
        // the copies land before the CTA goes away, whoever gave up
        const int64_t first = issued > Stages ? issued - Stages : 0;
        for (int64_t i = first; i < issued; ++i)
          mbar_wait(&full_bar[i % Stages], static_cast<uint32_t>((i / Stages) & 1), p.timeout_ns,
                    p.status);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp walks the loop, so that its values stay in uniform
      // registers, where the MMA wants them; one lane issues.
      const uint32_t issue = elect_one_lane();
      const uint64_t desc_a = smem_desc_sw128(smem_addr(smem + L::kOffA));
      const uint64_t desc_b = smem_desc_sw128(smem_addr(smem + L::kOffB));
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      while (ok && next_tile<Mode, BN, Split>(walk, p, off, pre, tile)) {
        for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
          // The operands are usually there before the buffer is: what the
          // buffer's release waits for comes after it, in as few steps as
          // can be.
          ok = warp_wait(&full_bar[stage], phase, p, abort_flag) &&
               warp_wait(&tmem_empty[buf], buf_phase ^ 1, p, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          mma_block(tmem_base + static_cast<uint32_t>(buf * BN),
                    desc_a + static_cast<uint64_t>(stage * (kStageA >> 4)),
                    desc_b + static_cast<uint64_t>(stage * (L::kTileB >> 4)), idesc,
                    smem_addr(&tmem_full[buf]), smem_addr(&empty_bar[stage]), issue);
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
      // the MMAs issued end before the tensor memory is freed
      if (issue) {
        tc_commit(drain_bar);
        mbar_wait(drain_bar, 0, p.timeout_ns, p.status);
      }
    } else if (warp == kScaleWarp || ColScale) {
      // -------------------------------------------------------------- scales
      // Groups lie at multiples of four K blocks: a tile's first may begin
      // before the tile; an empty segment has none.  The next group's column
      // scales are loaded before its place is free.
      const int part = warp - kScaleWarp;  // ColScale: this warp's half of the columns
      const uint64_t pol_scale = policy_evict_last();
      constexpr int kCols = ColScale ? BN / 64 : 1;  // per lane
      float4 v[kCols];
      int64_t groups = 0;
      int g = 0, kb = 0;
      uint32_t g_phase = 0;
      tile.kb1 = 0;
      auto next_group = [&]() {
        kb += kScaleGroup;
        while (kb >= tile.kb1) {
          if (!next_tile<Mode, BN, Split>(walk, p, off, pre, tile)) return false;
          kb = tile.kb0 < tile.kb1 ? tile.kb0 / kScaleGroup * kScaleGroup : tile.kb1;
        }
        if (ColScale) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            const int64_t col = min(tile.n0 + part * (BN / 2) + lane + 32 * j, p.N - 1);
            load_group(v[j], p.sb + col * p.lds_b, kb, tile.kb1, p.vec_b);
          }
        } else if (lane < 2 * kScaleGroup) {
          // lane = 4 half + K block of the group (past the last: the last)
          const int col = min(tile.n0 + lane / kScaleGroup * kHalf, p.N - 1);
          const int64_t block = col / kBlock;
          v[0].x = __ldg(p.sb + (Mode == Fp8Mode::kRows ? tile.expert * p.stride_sb : 0) +
                         block * p.lds_b + min(kb + lane % kScaleGroup, tile.kb1 - 1));
        }
        return true;
      };
      while (next_group()) {
        ok = warp_wait(&scale_empty[g], g_phase ^ 1, p, abort_flag);
        if (!ok) break;
        if (ColScale) {
          // [4][BN], a lane's columns 32 apart
          float* cs = col_scale + g * kScaleGroup * BN + part * (BN / 2) + lane;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            cs[32 * j] = v[j].x;
            cs[BN + 32 * j] = v[j].y;
            cs[2 * BN + 32 * j] = v[j].z;
            cs[3 * BN + 32 * j] = v[j].w;
          }
        } else if (lane < 2 * kScaleGroup) {
          col_scale[g * 2 * kScaleGroup + lane] = v[0].x;
        }
        uint8_t* rows = smem + L::kOffRow + g * kRowScaleBytes;
        if (part == 0 && !p.vec_a) {
          float4 r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t row = min(tile.row0 + lane + 32 * i, p.M - 1);
            load_group(r[i], p.sa + row * p.lds_a, kb, tile.kb1, 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(rows + (lane + 32 * i) * 16) = r[i];
        }
        __syncwarp();
        if (part == 0 && p.vec_a) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&scale_full[g], kRowScaleBytes);
            tma_load_2d(&tmap_sa, &scale_full[g], rows, kb, tile.row0, pol_scale);
          }
        } else {
          lane0_arrive(smem_addr(&scale_full[g]), lane);
        }
        ++groups;
        if (++g == 2) {
          g = 0;
          g_phase ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
      // the copies land before the CTA goes away
      for (int64_t i = groups > 2 ? groups - 2 : 0; i < groups; ++i)
        warp_wait(&scale_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), p, abort_flag);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    // ---------------------------------------------------- sums and epilogue
    const int in_tile = (warp & 3) * 32, half = warp >> 2;
    const uint32_t src0 =
        tmem_base + (static_cast<uint32_t>(in_tile) << 16) + static_cast<uint32_t>(half * kHalf);
    const uint32_t empty0 = smem_addr(&tmem_empty[0]);
    uint8_t* boxes = smem + L::kOffBox + warp * L::kBoxes * kBoxBytes;
    int buf = 0, g = 0, next_box = 0;
    uint32_t buf_phase = 0, g_phase = 0;
    while (ok && next_tile<Mode, BN, Split>(walk, p, off, pre, tile)) {
      float2 acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      // the warp's biases, on their way during the K blocks (32768 x 4096 x 2048
      // with bias and GELU: 299 us, loaded after them 307)
      float bias_ahead[kHalf / 32];
      if (Mode != Fp8Mode::kK && !Split && (p.flags & kEpiBias)) {
        const int64_t at = Mode == Fp8Mode::kRows ? tile.expert * p.stride_bias : 0;
#pragma unroll
        for (int c = 0; c < kHalf; c += 32)
          bias_ahead[c / 32] =
              load_as_f32(p.bias, at + min(tile.n0 + half * kHalf + c + lane, p.N - 1), p.dtype_d);
      }
      // the scales of a group of K blocks: the row's, and its half's weight block's
      float4 ra, ca;
#pragma unroll 1
      for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
        const int in_group = kb % kScaleGroup;
        if (in_group == 0 || kb == tile.kb0) {
          ok = warp_wait(&scale_full[g], g_phase, p, abort_flag);
          ra = *reinterpret_cast<const float4*>(smem + L::kOffRow + g * kRowScaleBytes +
                                                (in_tile + lane) * 16);
          if (!ColScale)
            ca = *reinterpret_cast<const float4*>(col_scale + (g * 2 + half) * kScaleGroup);
          else  // a segment's first block may lie inside a group
            for (int i = 0; i < in_group; ++i) ra = make_float4(ra.y, ra.z, ra.w, 0.0f);
        }
        const float* cs = col_scale + (g * kScaleGroup + in_group) * BN + half * kHalf;
        ok = ok && warp_wait(&tmem_full[buf], buf_phase, p, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t src = src0 + static_cast<uint32_t>(buf * BN);
        // 16 columns are loaded while the 16 before are added
        uint32_t v[2][16];
        tmem_ld_16cols(src, v[0]);
        const float s = ColScale ? ra.x : ra.x * ca.x;
        const float2 s2 = make_float2(s, s);
        ra = make_float4(ra.y, ra.z, ra.w, 0.0f);
        if (!ColScale) ca = make_float4(ca.y, ca.z, ca.w, 0.0f);
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
          uint32_t(&x)[16] = v[(c / 16) & 1];
          tc_wait_ld16(x);
          if (c + 16 < kHalf) {
            tmem_ld_16cols(src + c + 16, v[(c / 16 + 1) & 1]);
          } else {
            tc_fence_before_sync();
            __syncwarp();
            lane0_arrive(empty0 + static_cast<uint32_t>(buf * 8), lane);
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float2 t0 = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            float2 t1 = make_float2(__uint_as_float(x[2 * i + 2]), __uint_as_float(x[2 * i + 3]));
            if (ColScale) {
              const float4 k = *reinterpret_cast<const float4*>(cs + c + 2 * i);
              t0 = mul2(t0, make_float2(k.x, k.y));
              t1 = mul2(t1, make_float2(k.z, k.w));
            }
            acc[c / 2 + i] = fma2(t0, s2, acc[c / 2 + i]);
            acc[c / 2 + i + 1] = fma2(t1, s2, acc[c / 2 + i + 1]);
          }
        }
        if (++buf == kBufs) {
          buf = 0;
          buf_phase ^= 1;
        }
        if (in_group == kScaleGroup - 1 || kb + 1 == tile.kb1) {
          __syncwarp();  // every lane has its scales of the group
          lane0_arrive(smem_addr(&scale_empty[g]), lane);
          if (++g == 2) {
            g = 0;
            g_phase ^= 1;
          }
        }
      }
      if (!ok) break;
      int first = tile.n0 + half * kHalf, columns = kHalf;  // of D, for this warp to finish
      if (Split) {
        // Each CTA's sums go to its own shared memory (its stages are spent:
        // every MMA has been waited for), and each finishes its share of the
        // columns, adding the CTAs' sums in the order of K.
        columns = kHalf / p.split;
        const int skip = walk.rank * columns;
        first += skip;
        float4* mine = reinterpret_cast<float4*>(smem) + warp * (kHalf / 4) * 32 + lane;
#pragma unroll
        for (int i = 0; i < kHalf / 4; ++i)
          mine[i * 32] =
              make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
        cluster_sync();
        met = true;
        const uint32_t share = smem_addr(mine + skip / 4 * 32);
#pragma unroll
        for (int i = 0; i < kHalf / 8; ++i) {
          if (4 * i >= columns) break;
          float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int r = 0; r < p.split; ++r) {
            const float4 v = ld_cluster_float4(
                mapa_shared(share + static_cast<uint32_t>(i * 32 * 16), static_cast<uint32_t>(r)));
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
          }
          acc[2 * i] = make_float2(sum.x, sum.y);
          acc[2 * i + 1] = make_float2(sum.z, sum.w);
        }
      }
      // D, 32 columns at a time; the sums move down so that the loop's body
      // (whose GELU is long) is there once
      const int matrix = Mode == Fp8Mode::kK ? tile.expert : 0;
      const int64_t row = tile.row0 + min(in_tile + lane, tile.rows - 1);
      const int64_t drow = matrix * p.stride_d + row * p.ldd;
      const int64_t bias0 = Mode == Fp8Mode::kRows ? tile.expert * p.stride_bias : 0;
      const int col_end = tile.rows > in_tile ? min(p.N, first + columns) : 0;
      if (!Split && p.beta == 0.0f) {
        if (col_end == 0 || first >= p.N) continue;
        // Straight through all of the warp's columns, N's or not (experts' gradients
        // 527 us, were 687 in the loop below, 5900 clocks a tile; 2000^3, whose last
        // tiles are cut, 2 us less than with those in the loop).
        float2 alpha = make_float2(p.alpha, p.alpha);
        if (Mode != Fp8Mode::kK && (p.flags & kEpiBias)) {
          // the biases to all lanes, by way of a box (each lane loading all of
          // them, 16 columns at a time: 43 us more)
          float* bias = reinterpret_cast<float*>(boxes);
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) bias[c + lane] = bias_ahead[c / 32];
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kHalf; c += 4) {
            const float4 k = *reinterpret_cast<const float4*>(bias + c);
            acc[c / 2] = fma2(acc[c / 2], alpha, make_float2(k.x, k.y));
            acc[c / 2 + 1] = fma2(acc[c / 2 + 1], alpha, make_float2(k.z, k.w));
          }
          alpha = make_float2(1.0f, 1.0f);
          __syncwarp();
        }
        if (Mode != Fp8Mode::kK && (p.flags & kEpiGelu)) {
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) acc[i] = gelu2(mul2(acc[i], alpha));
          alpha = make_float2(1.0f, 1.0f);
        }
        auto pass = [&](auto columns_of_box, auto put) {
          constexpr int kCols = decltype(columns_of_box)::value;
#pragma unroll
          for (int c = 0; c < kHalf; c += kCols) {
            if (first + c >= p.N) break;
            uint8_t* box = boxes + next_box * kBoxBytes;
            if (++next_box == L::kBoxes) next_box = 0;
            if (lane == 0) bulk_wait_group_read<L::kBoxes - 1>();  // its last store has read it
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kBoxRow / 16; ++q)
              *reinterpret_cast<uint4*>(box + box_offset(lane, q)) =
                  put(c / 2 + q * (kCols * 16 / kBoxRow / 2));
            send_box(&tmap_d, box, p, tile, in_tile, first + c, kBoxRow / 16, matrix, lane);
          }
        };
        if (p.dtype_d == DG_F32)
          pass(std::integral_constant<int, 32>(), [&](int i) {
            const float2 x = mul2(acc[i], alpha), y = mul2(acc[i + 1], alpha);
            return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x),
                              __float_as_uint(y.y));
          });
        else if (p.dtype_d == DG_BF16)
          pass(std::integral_constant<int, 64>(), [&](int i) {
            return pack8<BF16>(mul2(acc[i], alpha), mul2(acc[i + 1], alpha),
                               mul2(acc[i + 2], alpha), mul2(acc[i + 3], alpha));
          });
        else
          pass(std::integral_constant<int, 64>(), [&](int i) {
            return pack8<F16>(mul2(acc[i], alpha), mul2(acc[i + 1], alpha),
                              mul2(acc[i + 2], alpha), mul2(acc[i + 3], alpha));
          });
        continue;
      }
      int fill = 0, box_col = 0;  // the open box: 16-byte pieces in it, its first column
#pragma unroll 1
      for (int col0 = first; col0 < col_end; col0 += 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = col0 + 16 * h;
          if (col >= col_end) break;
          float x[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[2 * i] = acc[8 * h + i].x;
            x[2 * i + 1] = acc[8 * h + i].y;
          }
          finish16<Mode>(x, p, drow, col, bias0);
          uint8_t* box = boxes + next_box * kBoxBytes;
          if (fill == 0) {
            box_col = col;
            if (lane == 0) bulk_wait_group_read<L::kBoxes - 1>();  // its last store has read it
            __syncwarp();
          }
          if (p.dtype_d == DG_F32) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(box + box_offset(lane, fill + q)) =
                  make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            fill += 4;
          } else {
            uint32_t w[8];
            if (p.dtype_d == DG_BF16) {
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = BF16::pack(x[2 * i], x[2 * i + 1]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = F16::pack(x[2 * i], x[2 * i + 1]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
              *reinterpret_cast<uint4*>(box + box_offset(lane, fill + q)) =
                  make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            fill += 2;
          }
          if (fill == kBoxRow / 16 || col + 16 >= col_end) {
            send_box(&tmap_d, box, p, tile, in_tile, box_col, fill, matrix, lane);
            fill = 0;
            if (++next_box == L::kBoxes) next_box = 0;
          }
        }
#pragma unroll
        for (int i = 0; i + 16 < kHalf / 2; ++i) acc[i] = acc[i + 16];
      }
    }
    if (!ok) *abort_flag = 1;
    if (lane == 0) bulk_wait_group<0>();  // this thread's stores end before the CTA does
  }
  __syncwarp();
  if (Split) {
    if (!met) cluster_sync();  // the sums are there
    cluster_sync();            // and have been read
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc<kTmemCols>(tmem_base);
  }
}

// The K blocks of each CTA of a split tile (the last may have fewer, or none):
// whole groups.
int share_of_k(int64_t k_blocks, int split) {
  const int64_t groups = (k_blocks + kScaleGroup - 1) / kScaleGroup;
  return static_cast<int>((groups + split - 1) / split * kScaleGroup);
}

template <Fp8Mode Mode, int BN, int Stages, bool ColScale, bool Split = false>
cudaError_t run_fp8(const Fp8Args& a, int split = 1) {
  using L = F8Smem<BN, Stages, ColScale>;
  // Fewer rows than a tile: only those (whole swizzle atoms of 8) are loaded;
  // the stale shared memory below feeds rows of D that are not there.
  const int box_a = Mode == Fp8Mode::kDense && a.M < kRowsPerCta
                        ? static_cast<int>((a.M + 7) / 8 * 8)
                        : kRowsPerCta;
  CUtensorMap ta, tb;
  cudaError_t e = tc::encode_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, a.M, a.K, a.lda,
                                    box_a, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int64_t b_pitch = Mode == Fp8Mode::kRows ? a.stride_b / a.ldb : 0;
  const int64_t b_rows = Mode == Fp8Mode::kRows ? (a.count - 1) * b_pitch + a.N : a.N;
  e = tc::encode_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, b_rows, a.K, a.ldb, BN, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  F8Params p;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.m_blocks = static_cast<int>((a.M + kRowsPerCta - 1) / kRowsPerCta);
  p.n_blocks = static_cast<int>((a.N + BN - 1) / BN);
  p.most_blocks = static_cast<uint32_t>(kMaxTiles / p.n_blocks);
  p.k_blocks = static_cast<int>((a.K + kBlock - 1) / kBlock);
  p.k_rows = static_cast<int>(a.K);
  const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_blocks *
                        (Mode == Fp8Mode::kK ? a.count : 1);
  p.tiles = static_cast<int>(std::min<int64_t>(tiles, INT32_MAX));
  p.split = split;
  p.split_blocks = share_of_k(p.k_blocks, split);
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
  p.vec_d = (a.ldd * z) % 16 == 0 && (a.stride_d * z) % 16 == 0 ? 1 : 0;
  // TMA clips a store at N in whole 16-byte pieces: another N would write past it
  p.tma_d = p.vec_d && (a.N * z) % 16 == 0 ? 1 : 0;
  auto vec = [](const float* s, int64_t ld, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(s) & 15) == 0 && ld % 4 == 0 && stride % 4 == 0;
  };
  p.vec_a = vec(a.sa, a.lds_a, 0);
  p.vec_b = vec(a.sb, a.lds_b, a.stride_sb);
  p.stage_tx = static_cast<uint32_t>(box_a * 128 + L::kTileB);
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  CUtensorMap td = ta;  // not used without tma_d
  if (p.tma_d) {
    e = make_out_map(&td, a.D, a.dtype_d, a.M, a.N, a.ldd, Mode == Fp8Mode::kK ? a.count : 1,
                     a.stride_d);
    if (e != cudaSuccess) return e;
  }

  CUtensorMap tsa = ta;  // not used without vec_a
  if (p.vec_a) {
    // whole groups: they end within the row's pitch, a multiple of four
    const int64_t width = (p.k_blocks + kScaleGroup - 1) / kScaleGroup * kScaleGroup;
    e = tc::encode_map_2d(&tsa, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.sa, a.M, width, a.lds_a * 4,
                          kRowsPerCta, kScaleGroup, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }

  auto kern = gemm_fp8_kernel<Mode, BN, Stages, ColScale, Split>;
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
                           ? (a.M / kRowsPerCta + std::min(a.count, a.M)) * p.n_blocks
                           : tiles;
  if (most > kMaxTiles) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
      Split ? most * split : std::max<int64_t>(1, std::min<int64_t>(most, a.sm_count))));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(L::bytes(p.count));
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = Split ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, td, tsa, p);
  count_launches(1);
  return e;
}

// 128 x 256 tiles, except where 128 x 128 tiles take no more rounds over the
// SMs: a K block of the narrow tile costs 0.6 of the wide one's time (4096^3, 512
// wide tiles or 1024 narrow: 65 us or 77; 2000^3, 128 or 256: 15.0 us or 17.5;
// 1000 x 2000 x 2000, 64 or 128: 18.0 us or 11.9).  A dense product's narrow
// tiles are split along K over clusters of four CTAs, or of two where there are
// not SMs for four, if that saves the longest share enough K blocks.  Shares are
// whole scale groups of four blocks, so the last may be shorter or empty.  A
// cluster costs about 5 us (its launch, two barriers, the sums' way through
// shared memory) in halves and 4 in quarters; a K block 0.28 us, with column
// scales 0.44.  Measured in us, whole / split:
//   halves, 64 x 8000 and 256 x 4096: K = 4096 (16 blocks saved) 12.7 / 13.0, 5120
//   (20) 15.1 / 14.2, 8192 (32) 22.2 / 17.9; column scales: K = 2816 (10) 13.4 /
//   13.8, 3584 (12) 15.8 / 15.6, 4096 (16) 17.8 / 15.7;
//   quarters, 64 x 4096: K = 2560 (12 saved) 8.9 / 9.3, 2816 (14) 9.6 / 9.3, 4096
//   (24) 12.5 / 9.6; column scales: K = 1536 (8) 8.4 / 9.0, 1792 (10) 9.4 / 9.0,
//   4096 (24) 17.5 / 11.2.
template <Fp8Mode Mode, bool ColScale>
cudaError_t run_shape(const Fp8Args& a) {
  const int64_t row_blocks = (Mode == Fp8Mode::kRows
                                  ? a.M / 128 + std::min(a.count, a.M)
                                  : (a.M + 127) / 128) *
                             (Mode == Fp8Mode::kK ? a.count : 1);
  auto rounds = [&](int64_t bn) {
    const int64_t tiles = row_blocks * ((a.N + bn - 1) / bn);
    return (tiles + a.sm_count - 1) / a.sm_count;
  };
  if (rounds(256) < rounds(128)) return run_fp8<Mode, 256, 3, ColScale>(a);
  if constexpr (Mode == Fp8Mode::kDense) {
    const int64_t tiles = row_blocks * ((a.N + 127) / 128);
    const int64_t k_blocks = (a.K + kBlock - 1) / kBlock;
    const int split = tiles * 4 <= a.sm_count ? 4 : 2;
    const int64_t saved = k_blocks - share_of_k(k_blocks, split);
    const int64_t enough = split == 4 ? (ColScale ? 10 : 14) : (ColScale ? 12 : 18);
    if (tiles * split <= a.sm_count && saved >= enough)
      return run_fp8<Mode, 128, 5, ColScale, true>(a, split);
  }
  return run_fp8<Mode, 128, 5, ColScale>(a);
}

}  // namespace

cudaError_t launch_fp8_tc(const Fp8Args& a) {
  switch (a.mode) {
    case Fp8Mode::kDense:
      return a.block_rows_b == 1 ? run_shape<Fp8Mode::kDense, true>(a)
                                 : run_shape<Fp8Mode::kDense, false>(a);
    case Fp8Mode::kRows: return run_shape<Fp8Mode::kRows, false>(a);
    case Fp8Mode::kK: return run_shape<Fp8Mode::kK, true>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dg
