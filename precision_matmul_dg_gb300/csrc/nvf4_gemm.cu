// Products of 4-bit operands with an E4M3 scale per 16 values and an FP32 scale
// per row (dg_gemm_nvf4, dg_gemm_nvf4_grouped in dg.h) on the block-scaled
// tcgen05 MMA (kind::mxf4nvf4, K = 64):
//
//   t[i,j] = ra[i] rb[j] * sum over k of  (a sa)[i,k] * (b sb)[j,k]
//
// The tensor core applies the blocks' scales itself and adds in FP32 in tensor
// memory over all of K; the rows' scales are two multiplications at the end.
//
//   warp 0       TMA producer of a ring of stages: 256 values of K (128 bytes)
//                of 128 rows of A and BN rows of B, and the scale tiles of both
//                (512 bytes for 128 rows and 64 values, stored as the copies
//                into tensor memory read them);
//   warp 1       MMA issuer: per stage the scale tiles go to one of two buffers
//                in tensor memory (tcgen05.cp, in order with the MMAs), then
//                four MMAs;
//   warp 2       tensor memory allocation;
//   warps 4 ..   epilogue, 64 columns x 32 rows each, from one of two
//                accumulators while the next tile is multiplied.
//
// CG = 2: CTA pairs on 256 x BN tiles, half of B's rows each, which halves B's
// share of the way from L2.  What bounds large products (8192^3 204 us; its MMAs
// alone, at four times the 16-bit rate, 143): MMAs and scale copies go through one
// queue (without the copies 173 us), and the operands from L2 alone take 156.
//
// Persistent: unit u (a CTA or a pair) takes tiles u, u + units, ...  Experts'
// rows are read from the device's offsets, multiples of 128 as the scale tiles
// are; a row tile may run into the next expert's rows (loaded, never stored).
#include <algorithm>

#include "epilogue.cuh"
#include "fp8.cuh"
#include "out_box.cuh"
#include "segments.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kStageK = 256;                    // values of K per stage
constexpr int kStageA = 128 * 128;              // bytes of codes
constexpr int kSfTile = 512;                    // 128 rows x 4 scales
constexpr int kSfBlock = 4 * kSfTile;           // of a stage, for 128 rows

struct N4Params {
  int M, N;
  int m_blocks, n_blocks, k_blocks, k_tiles;  // k_tiles: scale tiles along K
  int tiles, group_m, count;
  int b_rows;           // rows of B's map from one expert to the next
  int sfa_rows, sfb_rows;  // scale tile rows (128 rows each) of A, of one B
  const int32_t* offsets;
  uint32_t most_blocks;  // experts: row blocks whose tiles a walk takes
  const float *row_a, *row_b;
  void* D;
  int64_t ldd, stride_d;
  const void* bias;
  int64_t stride_bias;
  float alpha, beta;
  int flags, dtype_d;
  int tma_d, vec_d;
  uint32_t stage_tx;
  int* status;
  uint64_t timeout_ns;
};

template <int BN, int Stages, int CG>
struct N4Smem {
  static constexpr int kRowsB = BN / CG;
  static constexpr int kTileB = kRowsB * 128;
  static constexpr int kSfBlocksB = BN > 128 ? 2 : 1;  // a tile of 192 starts at 0 or 64 of 128
  static constexpr int kSfBytes = (1 + kSfBlocksB) * kSfBlock;
  static constexpr int kEpiWarps = 4 * (BN / 64);
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + Stages * kStageA;
  static constexpr int kOffSf = kOffB + Stages * kTileB;
  static constexpr int kOffBox = kOffSf + Stages * kSfBytes;
  static constexpr int kOffCol = kOffBox + kEpiWarps * kBoxBytes;  // [warp][2][64] floats
  static constexpr int kOffBar = kOffCol + kEpiWarps * 512;
  static constexpr int kBars = 2 * Stages + 5;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kOffGroups = (kOffAbort + 4 + 15) / 16 * 16;
  static constexpr int bytes(int64_t count) {
    return kOffGroups + 1024 + static_cast<int>(count > 0 ? 2 * (count + 1) * 4 : 0);
  }
  static_assert(kTileB % 1024 == 0 && kOffSf % 128 == 0 && kOffBox % 1024 == 0, "alignment");
};

// Rows row0 .. row0 + rows - 1 of A and D (of this CTA), columns from n0.
struct N4Tile {
  int row0, rows, n0, expert;
};
struct N4Walk {
  int t, expert;
};

template <bool Grouped, int BN, int CG>
__device__ __forceinline__ bool next_tile(N4Walk& w, const N4Params& p, int units, int rank,
                                          const int* off, const int* pre, N4Tile& o) {
  int m, nb, end;
  if (Grouped) {
    while (w.expert < p.count && w.t >= pre[w.expert + 1] * p.n_blocks) ++w.expert;
    if (w.expert >= p.count) return false;
    const int mb = pre[w.expert + 1] - pre[w.expert];
    const int local = w.t - pre[w.expert] * p.n_blocks;
    nb = local / mb;  // rows first: concurrent tiles share weights
    m = local - nb * mb;
    o.expert = w.expert;
    o.row0 = off[w.expert];
    end = off[w.expert + 1];
  } else {
    if (w.t >= p.tiles) return false;
    tc::tile_coords(w.t, p.m_blocks, p.n_blocks, p.group_m, m, nb);
    o.expert = 0;
    o.row0 = 0;
    end = p.M;
  }
  o.row0 += (m * CG + rank) * 128;
  o.rows = min(128, end - o.row0);  // none or negative: the pair's second half lies past the end
  o.n0 = nb * BN;
  w.t += units;
  return true;
}

// A warp's 64 columns of an accumulator times its rows' factors s (alpha times a row scale)
// and the columns' scales `col`, in place: what the epilogue does on its way, for tiles with
// a row whose s is outside [2^-100, 2^65).  Such an s is s1 g, s1 between 2^-104 and 2^65
// and g a power of two: a nonzero sum of codes times scales is between 2^-20 and 2^53 in
// magnitude, so sum * s1 is in FP32's normal range, and sum * s1 * (a column's scale) leaves
// it only where the result does too: g then moves it further out.
//   Ahead of the epilogue, which is as it was: 32768 x 4096 x 2048 with bias and GELU 141.6
// us, with g in the epilogue 147.6, with a copy of it 143.4.
constexpr uint32_t kNearExp = 127 - 100, kFarExp = 127 + 64;
__device__ __forceinline__ void scale_far(uint32_t taddr, float s, const float* col) {
  const uint32_t e = __float_as_uint(s) >> 23 & 0xFFu;
  float g = 1.0f;
  if (e > kFarExp && e < 255) {  // to 2^64 .. 2^65
    g = __uint_as_float((e - kFarExp + 127) << 23);
    s = __uint_as_float((__float_as_uint(s) & 0x807FFFFFu) | kFarExp << 23);
  } else if (e < kNearExp) {  // below 2^-100, subnormal ones too
    g = 0x1p-45f;
    s *= 0x1p45f;
  }
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    uint32_t x[32];
    tmem_ld_32cols(taddr + static_cast<uint32_t>(c), x);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      x[i] = __float_as_uint(__uint_as_float(x[i]) * s * col[c + i] * g);
    tc::tmem_st_32cols(taddr + static_cast<uint32_t>(c), x);
  }
  tc::tc_wait_st();
  __syncwarp();  // `col` has been read
}

template <bool Grouped, int BN, int Stages, int CG>
__global__ void __launch_bounds__((4 + 4 * (BN / 64)) * 32, 1)
    gemm_nvf4_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_sfa,
                     const __grid_constant__ CUtensorMap tmap_sfb,
                     const __grid_constant__ CUtensorMap tmap_d,
                     const __grid_constant__ N4Params p) {
  using L = N4Smem<BN, Stages, CG>;
  constexpr int kThreads = (4 + L::kEpiWarps) * 32;
  // two accumulators, then two buffers of scale words: per word (64 values) 4
  // columns for A's 128 rows and 4 for each 128 rows of B
  constexpr int kSfColsB = 4 * L::kSfBlocksB;  // per word
  constexpr int kSfCols = 4 * (4 + kSfColsB);
  constexpr int kColsNeeded = 2 * BN + 2 * kSfCols;
  constexpr int kTmemCols = kColsNeeded <= 256 ? 256 : 512;
  static_assert(kColsNeeded <= 512, "tensor memory");
  constexpr uint32_t idesc = idesc_nvf4(128 * CG, BN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty_bar = full_bar + Stages;
  uint64_t* tmem_full = empty_bar + Stages;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* drain_bar = tmem_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  int* off = reinterpret_cast<int*>(smem + L::kOffGroups);
  int* pre = off + p.count + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / CG, units = static_cast<int>(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], CG * L::kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
    tma_prefetch_desc(&tmap_sfa);
    tma_prefetch_desc(&tmap_sfb);
    tma_prefetch_desc(&tmap_d);
  }
  if (warp == 2) {
    if (CG == 2)
      tmem_alloc_pair<kTmemCols>(tmem_slot);
    else
      tmem_alloc<kTmemCols>(tmem_slot);
  }
  // Launched as a programmatic dependent: everything above is the CTA's own
  // on-chip state; global memory waits for the kernel before.
  grid_dependency_wait();
  if (Grouped) {
    // offsets clamped to the rows there are, down to whole tiles of 128
    bool odd = false;
    for (int e = threadIdx.x; e <= p.count; e += kThreads) {
      const int v = min(max(__ldg(p.offsets + e), 0), p.M);
      const bool whole = (v & 127) == 0 || v == p.M;
      odd |= !whole;
      off[e] = whole ? v : v & ~127;
    }
    if (odd && blockIdx.x == 0) atomicExch(p.status, static_cast<int>(DG_ERR_INVALID_ARG));
    __syncthreads();
    if (warp == 3)
      count_row_blocks(off, pre, p.count, 128 * CG, p.most_blocks, blockIdx.x == 0, p.status, lane);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the peer's barriers are there before any remote arrival
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;
  N4Walk walk{unit, 0};
  N4Tile tile;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one_lane()) {
      const uint64_t pol = policy_evict_last();  // tiles are read again by other CTAs
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      while (ok && next_tile<Grouped, BN, CG>(walk, p, units, rank, off, pre, tile)) {
        const int b_row = tile.expert * p.b_rows + tile.n0 + rank * L::kRowsB;
        // scale tiles past the last: any that is there (their rows are not stored)
        const int sfa = min(tile.row0 >> 7, p.sfa_rows - 1) * p.k_tiles;
        const int sb0 = tile.n0 >> 7;
        const int sfb = (tile.expert * p.sfb_rows + sb0) * p.k_tiles;
        const int sfb2 = (tile.expert * p.sfb_rows + min(sb0 + 1, p.sfb_rows - 1)) * p.k_tiles;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status,
                                   abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* dst_a = smem + L::kOffA + stage * kStageA;
          uint8_t* dst_b = smem + L::kOffB + stage * L::kTileB;
          uint8_t* dst_s = smem + L::kOffSf + stage * L::kSfBytes;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], p.stage_tx);
          if (CG == 1) {
            uint64_t* bar = &full_bar[stage];
            tma_load_2d(&tmap_a, bar, dst_a, kb * 128, tile.row0, pol);
            tma_load_2d(&tmap_b, bar, dst_b, kb * 128, b_row, pol);
            tma_load_2d(&tmap_sfa, bar, dst_s, 0, sfa + 4 * kb, pol);
            tma_load_2d(&tmap_sfb, bar, dst_s + kSfBlock, 0, sfb + 4 * kb, pol);
            if (L::kSfBlocksB == 2)
              tma_load_2d(&tmap_sfb, bar, dst_s + 2 * kSfBlock, 0, sfb2 + 4 * kb, pol);
          } else {
            // both CTAs' copies complete on the even CTA's barrier; each CTA
            // holds all of B's scales, as the MMA reads them in both
            const uint32_t bar = mapa_shared(smem_addr(&full_bar[stage]), 0);
            tma_load_2d_pair(&tmap_a, bar, dst_a, kb * 128, tile.row0, pol);
            tma_load_2d_pair(&tmap_b, bar, dst_b, kb * 128, b_row, pol);
            tma_load_2d_pair(&tmap_sfa, bar, dst_s, 0, sfa + 4 * kb, pol);
            tma_load_2d_pair(&tmap_sfb, bar, dst_s + kSfBlock, 0, sfb + 4 * kb, pol);
            if (L::kSfBlocksB == 2)
              tma_load_2d_pair(&tmap_sfb, bar, dst_s + 2 * kSfBlock, 0, sfb2 + 4 * kb, pol);
          }
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
      for (int64_t i = first; i < issued && leader; ++i)
        mbar_wait(&full_bar[i % Stages], static_cast<uint32_t>((i / Stages) & 1), p.timeout_ns,
                  p.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && elect_one_lane()) {
      int stage = 0, acc = 0, sf_buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      while (ok && next_tile<Grouped, BN, CG>(walk, p, units, rank, off, pre, tile)) {
        if (!mbar_wait_abortable(&tmem_empty[acc], acc_phase ^ 1, p.timeout_ns, p.status,
                                 abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        // a tile whose first column is 64 past a scale tile's starts 2 columns
        // into that tile's words
        const uint32_t sfb_skip = static_cast<uint32_t>((tile.n0 & 127) >> 5);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait_abortable(&full_bar[stage], phase, p.timeout_ns, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t da = smem_desc_sw128(smem_addr(smem + L::kOffA + stage * kStageA));
          const uint64_t db = smem_desc_sw128(smem_addr(smem + L::kOffB + stage * L::kTileB));
          const uint32_t src = smem_addr(smem + L::kOffSf + stage * L::kSfBytes);
          const uint32_t sfa_t = tmem_base + static_cast<uint32_t>(2 * BN + sf_buf * kSfCols);
          const uint32_t sfb_t = sfa_t + 16;
          // words past the last scale tile are another's: their codes are zero,
          // but a NaN among them would not be
          const int words = min(4, p.k_tiles - 4 * kb);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (w >= words) break;
            const uint64_t sa = smem_desc_rows16(src + w * kSfTile);
            if (CG == 2)
              tc_cp_32x128b_warpx4_pair(sfa_t + 4 * w, sa);
            else
              tc_cp_32x128b_warpx4(sfa_t + 4 * w, sa);
#pragma unroll
            for (int h = 0; h < L::kSfBlocksB; ++h) {
              const uint64_t sb = smem_desc_rows16(src + (1 + h) * kSfBlock + w * kSfTile);
              const uint32_t to = sfb_t + static_cast<uint32_t>(kSfColsB * w + 4 * h);
              if (CG == 2)
                tc_cp_32x128b_warpx4_pair(to, sb);
              else
                tc_cp_32x128b_warpx4(to, sb);
            }
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (w >= words) break;
            // 64 values are 32 bytes further into the swizzled rows
            tc_mma_nvf4<CG>(d_tmem, da + 2 * w, db + 2 * w, idesc, sfa_t + 4 * w,
                            sfb_t + static_cast<uint32_t>(kSfColsB * w) + sfb_skip,
                            (kb != 0 || w != 0) ? 1u : 0u);
          }
          sf_buf ^= 1;
          if (CG == 2)
            tc_commit_pair_multicast(&empty_bar[stage], 0x3);
          else
            tc_commit(&empty_bar[stage]);
          if (++stage == Stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (CG == 2)
          tc_commit_pair_multicast(&tmem_full[acc], 0x3);
        else
          tc_commit(&tmem_full[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
      // the MMAs issued end before the tensor memory is freed
      if (CG == 2)
        tc_commit_pair(drain_bar);
      else
        tc_commit(drain_bar);
      mbar_wait(drain_bar, 0, p.timeout_ns, p.status);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // A warp reads TMEM lanes 32 * (warp % 4) .. +31 only; each takes 64 columns.
    const int wi = warp - 4;
    const int in_tile = (wi & 3) * 32, first = (wi >> 2) * 64;
    const uint32_t empty0 =
        CG == 2 ? mapa_shared(smem_addr(&tmem_empty[0]), 0) : smem_addr(&tmem_empty[0]);
    uint8_t* box = smem + L::kOffBox + wi * kBoxBytes;
    float* col = reinterpret_cast<float*>(smem + L::kOffCol) + wi * 128;  // scales, then biases
    const int box_cols = p.dtype_d == DG_F32 ? 32 : 64;
    int acc = 0;
    uint32_t acc_phase = 0;
    // a tile's row scale, and the column scales and biases of two columns a lane,
    // loaded a tile ahead
    float row_next = 0.0f, col_next[2] = {0.0f, 0.0f}, bias_next[2] = {0.0f, 0.0f};
    auto load_ahead = [&]() {
      if (!next_tile<Grouped, BN, CG>(walk, p, units, rank, off, pre, tile)) return false;
      row_next = __ldg(p.row_a + min(tile.row0 + in_tile + lane, p.M - 1));
      const float* rb = p.row_b + static_cast<int64_t>(tile.expert) * p.N;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = min(tile.n0 + first + 32 * i + lane, p.N - 1);
        col_next[i] = __ldg(rb + c);
        if (p.flags & kEpiBias)
          bias_next[i] = load_as_f32(p.bias, tile.expert * p.stride_bias + c, p.dtype_d);
      }
      return true;
    };
    bool more = load_ahead();
    while (ok && more) {
      const N4Tile now = tile;
      const int col0 = now.n0 + first;
      const int row = min(now.row0 + in_tile + lane, p.M - 1);
      float s = p.alpha * row_next;
      // (see scale_far: zero, infinite and NaN factors go that way too)
      const bool far = __any_sync(
          0xffffffffu, (__float_as_uint(s) >> 23 & 0xFFu) - kNearExp > kFarExp - kNearExp);
      __syncwarp();  // the last tile's have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        col[32 * i + lane] = col_next[i];
        if (p.flags & kEpiBias) col[64 + 32 * i + lane] = bias_next[i];
      }
      __syncwarp();
      more = load_ahead();
      const bool got = mbar_wait_abortable(&tmem_full[acc], acc_phase, p.timeout_ns, p.status,
                                           abort_flag);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t src = tmem_base + (static_cast<uint32_t>(in_tile) << 16) +
                           static_cast<uint32_t>(acc * BN + first);
      const bool stored = now.rows > in_tile && col0 < p.N;
      const int64_t drow = static_cast<int64_t>(row) * p.ldd;
      if (far) {
        scale_far(src, s, col);
        s = 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) col[32 * i + lane] = 1.0f;
        __syncwarp();
      }
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        uint32_t x[32];
        tmem_ld_32cols(src + static_cast<uint32_t>(c), x);
        tc_wait_ld();
        if (c == 32) {  // all of the warp's columns are in registers
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            // (a cluster-scope release would wait for the warp's stores: there is
            // nothing in memory to release)
            if (CG == 2)
              mbar_arrive_remote(empty0 + static_cast<uint32_t>(acc * 8));
            else
              mbar_arrive(&tmem_empty[acc]);
          }
        }
        if (!stored || col0 + c >= p.N) continue;
        float2 v[16];
        const float2 s2 = make_float2(s, s);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float4 k = *reinterpret_cast<const float4*>(col + c + 2 * i);
          v[i] = mul2(mul2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                           s2),
                      make_float2(k.x, k.y));
          v[i + 1] = mul2(mul2(make_float2(__uint_as_float(x[2 * i + 2]),
                                           __uint_as_float(x[2 * i + 3])),
                               s2),
                          make_float2(k.z, k.w));
        }
        if (p.beta != 0.0f) {
          const int64_t z = p.dtype_d == DG_F32 ? 4 : 2;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[2 * i] = v[8 * h + i].x, t[2 * i + 1] = v[8 * h + i].y;
            add16(t, p.beta,
                  static_cast<const uint8_t*>(p.D) + (drow + col0 + c + 16 * h) * z, p.dtype_d,
                  p.N - (col0 + c + 16 * h));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * h + i] = make_float2(t[2 * i], t[2 * i + 1]);
          }
        }
        if (p.flags & kEpiBias) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 k = *reinterpret_cast<const float2*>(col + 64 + c + 2 * i);
            v[i] = make_float2(v[i].x + k.x, v[i].y + k.y);
          }
        }
        if (p.flags & kEpiGelu) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = gelu2(v[i]);
        }
        if (c == 0 || box_cols == 32) {
          if (lane == 0) bulk_wait_group_read<0>();  // the box's last store has read it
          __syncwarp();
        }
        if (p.dtype_d == DG_F32) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(box + box_offset(lane, q)) =
                make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
        } else if (p.dtype_d == DG_BF16) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(box + box_offset(lane, c / 8 + q)) =
                pack8<BF16>(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(box + box_offset(lane, c / 8 + q)) =
                pack8<F16>(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        // the box is full, or ends with D
        if (box_cols == 32)
          send_box(&tmap_d, box, p, now, in_tile, col0 + c, 8, 0, lane);
        else if (c == 32 || col0 + 32 >= p.N)
          send_box(&tmap_d, box, p, now, in_tile, col0, c == 32 ? 8 : 4, 0, lane);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (!ok) *abort_flag = 1;
    if (lane == 0) bulk_wait_group<0>();  // this thread's stores end before the CTA does
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (CG == 2) {
    if (*abort_flag) {
      // copies that the peer issued against this pair's barriers may still be
      // in flight after an abort
      if (threadIdx.x == 0) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 100000) sleep_ns(1000);
      }
      __syncthreads();
    }
    cluster_sync();  // the peer no longer reads this CTA's shared memory or barriers
  }
  if (warp == 2) {
    tc_fence_after_sync();
    if (CG == 2)
      tmem_dealloc_pair<kTmemCols>(tmem_base);
    else
      tmem_dealloc<kTmemCols>(tmem_base);
  }
}

template <bool Grouped, int BN, int Stages, int CG>
cudaError_t run_nvf4(const Nvf4Args& a) {
  using L = N4Smem<BN, Stages, CG>;
  constexpr int kMaxSmem = 227 * 1024;
  static_assert(L::bytes(0) <= kMaxSmem, "shared memory of a CTA");
  if (Grouped && L::bytes(a.count) > kMaxSmem) return cudaErrorInvalidValue;
  // Fewer rows than a tile: only those (whole swizzle atoms of 8) are loaded;
  // the stale shared memory below feeds rows of D that are not there.
  const int box_a =
      !Grouped && CG == 1 && a.M < 128 ? static_cast<int>((a.M + 7) / 8 * 8) : 128;
  const int64_t k_bytes = (a.K + 1) / 2;
  CUtensorMap ta, tb, tsa, tsb;
  cudaError_t e = tc::encode_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, a.M, k_bytes, a.lda,
                                    box_a, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int64_t b_pitch = Grouped ? a.stride_b / a.ldb : 0;
  const int64_t b_rows = Grouped ? (a.count - 1) * b_pitch + a.N : a.N;
  e = tc::encode_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, b_rows, k_bytes, a.ldb,
                        L::kRowsB, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  N4Params p;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.m_blocks = static_cast<int>((a.M + 128 * CG - 1) / (128 * CG));
  p.n_blocks = static_cast<int>((a.N + BN - 1) / BN);
  p.most_blocks = static_cast<uint32_t>(kMaxTiles / p.n_blocks);
  p.k_blocks = static_cast<int>((a.K + kStageK - 1) / kStageK);
  p.k_tiles = static_cast<int>((a.K + 63) / 64);
  const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_blocks;
  p.tiles = static_cast<int>(std::min<int64_t>(tiles, INT32_MAX));
  p.group_m = 16 / CG;
  p.count = Grouped ? static_cast<int>(a.count) : 0;
  p.b_rows = static_cast<int>(b_pitch);
  p.sfa_rows = static_cast<int>((a.M + 127) / 128);
  p.sfb_rows = static_cast<int>((a.N + 127) / 128);
  // scale tiles as rows of 512 bytes; a stage's four tiles of 128 rows follow
  // one another (past the matrix's last, what follows is loaded, not used)
  e = tc::encode_map_2d(&tsa, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.sa,
                        static_cast<int64_t>(p.sfa_rows) * p.k_tiles, 128, kSfTile, 4, 128,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  e = tc::encode_map_2d(&tsb, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.sb,
                        static_cast<int64_t>(p.sfb_rows) * p.k_tiles * (Grouped ? a.count : 1),
                        128, kSfTile, 4, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  p.offsets = a.offsets;
  p.row_a = a.row_a;
  p.row_b = a.row_b;
  p.D = a.D;
  p.ldd = a.ldd;
  p.stride_d = 0;
  p.bias = a.bias;
  p.stride_bias = a.stride_bias;
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.flags = a.epi;
  p.dtype_d = static_cast<int>(a.dtype_d);
  const int64_t z = a.dtype_d == DG_F32 ? 4 : 2;
  p.vec_d = (a.ldd * z) % 16 == 0 ? 1 : 0;
  // TMA clips a store at N in whole 16-byte pieces: another N would write past it
  p.tma_d = p.vec_d && (a.N * z) % 16 == 0 ? 1 : 0;
  p.stage_tx = static_cast<uint32_t>(CG * (box_a * 128 + L::kTileB + L::kSfBytes));
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  CUtensorMap td = ta;  // not used without tma_d
  if (p.tma_d) {
    e = make_out_map(&td, a.D, a.dtype_d, a.M, a.N, a.ldd, 1, 0);
    if (e != cudaSuccess) return e;
  }

  auto kern = gemm_nvf4_kernel<Grouped, BN, Stages, CG>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  static int max_units[64] = {};
  const int64_t most =
      Grouped ? (a.M / (128 * CG) + std::min(a.count, a.M)) * p.n_blocks : tiles;
  if (most > kMaxTiles) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((4 + L::kEpiWarps) * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(L::bytes(p.count));
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  e = once_per_device(attr_set, dev, [&]() {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSmem);
    if (r != cudaSuccess) return r;
    int n = a.sm_count / CG;
    if (CG == 2) {
      // pairs that fit at once
      cfg.numAttrs = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(a.sm_count & ~1));
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = a.sm_count / 2;
      }
    }
    max_units[dev & 63] = n;
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 2;
  const int64_t units = std::max<int64_t>(1, std::min<int64_t>(most, max_units[dev & 63]));
  cfg.gridDim = dim3(static_cast<unsigned>(units * CG));
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, tsa, tsb, td, p);
  count_launches(1);
  return e;
}

}  // namespace

// Which tile.  A stage takes a unit 0.34 us with 256 x 192 (pairs: half as many units),
// 0.30 with 128 x 128 and 0.29 with 128 x 64 (the scales' copies and the rows of A cost
// the same for fewer columns), so what counts is the number of rounds of tiles, weighted
// by that.  In us, pairs / 128 / 64:
//   16 x 8192 x 8192   19.4 / 13.8 / 13.3      256 x 4096 x 4096   10.8 / 9.2 / 8.5
//   256 x 8192 x 8192  17.0 / 14.8 / 22.6      1024 x 8192 x 8192  37.6 / 42.7 / 69.5
//   1024 x 4096 x 4096 16.9 / 14.4 / 23.2      2048 x 4096 x 4096  22.7 / 24.4 / 38.1
// Experts' row blocks are known on the device only, and a pair's second half may be
// empty: pairs from 512 rows per expert, of those that the caller makes room for.  64
// experts, 4096 x 2048, GELU, us, pairs / 128: all experts of 256 rows 87 / 96, 384 146 /
// 135, 512 150 / 175, 640 207 / 214, 1024 276 / 336; rows spread by half to either side,
// room for 312 each 112 / 113, 472 156 / 162, 578 176 / 194, 678 203 / 227, 1048 299 / 342.
cudaError_t launch_gemm_nvf4(const Nvf4Args& a) {
  const bool grouped = a.offsets != nullptr;
  auto cost = [&](int64_t row_blocks, int64_t cols, int64_t units, int64_t weight) {
    return (row_blocks * ((a.N + cols - 1) / cols) + units - 1) / units * weight;
  };
  const int64_t blocks = grouped ? a.M / 128 + std::min(a.count, a.M) : (a.M + 127) / 128;
  const int64_t c128 = cost(blocks, 128, a.sm_count, 30), c64 = cost(blocks, 64, a.sm_count, 29);
  if (grouped && a.M >= 512 * a.count) {
    // a fifth stage where the experts' table leaves room (up to 239 of them; 4096 tokens,
    // 8 of 64 experts, GELU: 179.5 us, with four 188.4)
    return N4Smem<192, 5, 2>::bytes(a.count) <= 227 * 1024 ? run_nvf4<true, 192, 5, 2>(a)
                                                          : run_nvf4<true, 192, 4, 2>(a);
  }
  if (!grouped && cost((a.M + 255) / 256, 192, a.sm_count / 2, 34) < std::min(c128, c64))
    return run_nvf4<false, 192, 5, 2>(a);
  if (c128 < c64) return grouped ? run_nvf4<true, 128, 5, 1>(a) : run_nvf4<false, 128, 5, 1>(a);
  return grouped ? run_nvf4<true, 64, 6, 1>(a) : run_nvf4<false, 64, 6, 1>(a);
}

}  // namespace dg
