// FP8 (E4M3) product with block scales for few rows (dg_gemm_fp8,
// dg_gemm_fp8_grouped with few rows per expert):
//   D[m,n] = epilogue(alpha * sum over blocks b of sa[m,b] * sb[n,b] *
//            sum over k in b of A[m,k] * B[n,k] + beta * D[m,n])
//
// The job is to stream N * K bytes of weights; each is used once or a few
// times.  A persistent CTA per SM keeps a ring of stages in shared memory full
// across its tiles, a stage being a few 128-byte blocks of K of the tile's
// weight rows and of 8 NT activation rows, loaded by TMA: up to 190 KB of loads
// are in flight per SM, whatever the warps do.  (16 x 8192 x 8192: 16.7 us;
// loads into registers that each warp waits for 29.5 us, one bulk copy per row
// and stage of 512 bytes 61 us.)
//
// Warps 0-7 multiply: warp-level m16n8k32 E4M3 MMAs, 16 weight rows as the
// one operand, 8 activation rows as the other.  The order of K inside a block
// is free as long as both operands share it, so a lane's fragments are 16-byte
// pieces of its rows: lane (g = lane / 4, q = lane % 4) holds bytes 64 h + 16 q
// .. + 15 of its rows for the two halves h of a 128-byte block, words 2 s and
// 2 s + 1 of a piece going to MMA step s.  Row g of an MMA is row g / 2 + 4 (g
// % 2) of the eight in memory: the rows that eight lanes read together then
// have their pieces, in the 128-byte swizzle, in different banks.
// Four MMAs make a block's sums, which then take the block's scales in FP32.
// Warp w takes row group w % RG of the tile and every (8 / RG)-th block; the
// groups' partial sums meet in shared memory in a fixed order (bit-stable).
//
// Tiles have 64, 32 or 16 weight rows: the largest of which there are enough
// for half the SMs.  Rows of several experts and more than 8 NT rows of one are
// further tiles, an expert's row chunks next to one another.
#include <algorithm>

#include "epilogue.cuh"
#include "fp8.cuh"
#include "segments.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kMmaWarps = 8;
constexpr int kThreads = (kMmaWarps + 1) * 32;

struct SkinnyParams {
  const float* sa;
  int64_t lds_a;
  const float* sb;
  int64_t lds_b, stride_sb;
  const int32_t* offsets;  // NULL: one product over M rows
  uint32_t most_blocks;  // experts: row blocks whose tiles a walk takes
  void* D;
  int64_t ldd;
  const void* bias;
  int64_t stride_bias;
  float alpha, beta;
  int M, N, K, count, flags, dtype_d, block_rows_b;
  int tiles_n, k_stages;  // tiles of weight rows; stages per tile
  int b_rows;             // rows of B's map from one expert to the next
  int* status;
  uint64_t timeout_ns;
};

template <int NT, int RG>
struct SkinnySmem {
  static constexpr int kSlices = kMmaWarps / RG;
  static constexpr int kBlocks = RG == 1 ? 1 : 2;         // per warp and stage
  static constexpr int kStageBlocks = kBlocks * kSlices;  // of K
  static constexpr int kRowsW = 16 * RG, kRowsX = 8 * NT;
  static constexpr int kBlockBytes = (kRowsW + kRowsX) * kBlock;
  static constexpr int kStage = kStageBlocks * kBlockBytes;
  static constexpr int kRed = 2 * kMmaWarps * NT * 4 * 32 * 4;
  static constexpr int kGroups = static_cast<int>(2 * (kMaxExperts + 1) * 4);
  static constexpr int kFree = 226 * 1024 - kRed - 256 - kGroups;  // 1 KB to align the base
  static constexpr int kStages = kFree / kStage < 8 ? kFree / kStage : 8;
  static_assert(kStages >= 2, "ring");
  static constexpr int kOffRed = kStages * kStage;
  static constexpr int kOffBar = kOffRed + kRed;
  static constexpr int kOffGroups = kOffBar + 256;
  static constexpr int bytes(int64_t count) {
    return 1024 + kOffGroups + static_cast<int>(count > 0 ? 2 * (count + 1) * 4 : 0);
  }
};

// A block's scales for one lane: of its two weight rows, of its two columns'
// activation rows.
template <int NT>
struct BlockScales {
  float a, b, x[NT][2];
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

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == DG_F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == DG_BF16 ? BF16::one(h) : F16::one(h);
}

// One tile: weight rows from n0 on, rows [m0, m1) of A and D.
struct SkinnyTile {
  int n0, m0, m1, expert;
};
struct SkinnyWalk {
  int t, expert;
};
// `off` and `pre`: the experts' row offsets and running chunk counts.
template <int NT, int RG>
__device__ __forceinline__ bool next_tile(SkinnyWalk& w, const SkinnyParams& p, const int* off,
                                          const int* pre, SkinnyTile& o) {
  int n, chunk, row0 = 0, row1 = p.M;
  o.expert = 0;
  if (p.offsets) {
    while (w.expert < p.count && w.t >= pre[w.expert + 1] * p.tiles_n) ++w.expert;
    if (w.expert >= p.count) return false;
    const int chunks = pre[w.expert + 1] - pre[w.expert];
    const int local = w.t - pre[w.expert] * p.tiles_n;
    n = local / chunks;
    chunk = local - n * chunks;
    row0 = off[w.expert];
    row1 = off[w.expert + 1];
    o.expert = w.expert;
  } else {
    const int chunks = (p.M + 8 * NT - 1) / (8 * NT);
    if (w.t >= chunks * p.tiles_n) return false;
    n = w.t / chunks;
    chunk = w.t - n * chunks;
  }
  o.n0 = n * 16 * RG;
  o.m0 = row0 + chunk * 8 * NT;
  o.m1 = min(row1, o.m0 + 8 * NT);
  w.t += static_cast<int>(gridDim.x);
  return true;
}

template <int NT, int RG>
__global__ void __launch_bounds__(kThreads, 1)
    skinny_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                      const __grid_constant__ CUtensorMap tmap_b,
                      const __grid_constant__ SkinnyParams p) {
  using L = SkinnySmem<NT, RG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + L::kOffRed);  // [2][warp][4 NT][lane]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty_bar = full_bar + L::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty_bar + L::kStages);
  int* off = reinterpret_cast<int*>(smem + L::kOffGroups);
  int* pre = off + p.count + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kMmaWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();  // launched as a dependent of the previous kernel
  if (p.offsets) {
    for (int e = threadIdx.x; e <= p.count; e += kThreads)
      off[e] = min(max(__ldg(p.offsets + e), 0), p.M);
    __syncthreads();
    if (warp == 0)
      count_row_blocks(off, pre, p.count, 8 * NT, p.most_blocks, blockIdx.x == 0, p.status, lane);
  }
  __syncthreads();
  SkinnyWalk walk{static_cast<int>(blockIdx.x), 0};
  SkinnyTile tile;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  const int blocks = (p.K + kBlock - 1) / kBlock;

  if (warp == kMmaWarps) {
    // ------------------------------------------------------------ producer
    if (!elect_one_lane()) return;
    const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
    int64_t issued = 0;
    while (ok && next_tile<NT, RG>(walk, p, off, pre, tile)) {
      const int b_row = tile.expert * p.b_rows + tile.n0;
      for (int ks = 0; ks < p.k_stages; ++ks) {
        ok = mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status, abort_flag);
        if (!ok) break;
        const int b0 = ks * L::kStageBlocks;
        const int n = min(L::kStageBlocks, blocks - b0);
        mbar_arrive_expect_tx(&full_bar[stage], static_cast<uint32_t>(n * L::kBlockBytes));
        uint8_t* dst = smem + stage * L::kStage;
        for (int j = 0; j < n; ++j, dst += L::kBlockBytes) {
          tma_load_2d(&tmap_b, &full_bar[stage], dst, (b0 + j) * kBlock, b_row, stream);
          tma_load_2d(&tmap_a, &full_bar[stage], dst + L::kRowsW * kBlock, (b0 + j) * kBlock,
                      tile.m0, keep);
        }
        ++issued;
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    grid_launch_dependents();
    if (!ok) *abort_flag = 1;
    // the copies land before the CTA goes away, whoever gave up
    const int64_t first = issued > L::kStages ? issued - L::kStages : 0;
    for (int64_t i = first; i < issued; ++i)
      mbar_wait(&full_bar[i % L::kStages], static_cast<uint32_t>((i / L::kStages) & 1),
                p.timeout_ns, p.status);
    return;
  }
  // ------------------------------------------------------------------- MMAs
  const int g = lane >> 2, q = lane & 3;
  const int group = warp % RG, slice = warp / RG;
  auto row_of = [](int i) { return (i >> 1) | ((i & 1) << 2); };
  const int gr = row_of(g);
  int turn = 0;
  while (next_tile<NT, RG>(walk, p, off, pre, tile)) {
    // rows past the last: their results are not stored
    const int na = min(tile.n0 + group * 16 + gr, p.N - 1);
    const int nb = min(tile.n0 + group * 16 + gr + 8, p.N - 1);
    const float* sb = p.sb + tile.expert * p.stride_sb;
    const float* sba = sb + static_cast<int64_t>(na / p.block_rows_b) * p.lds_b;
    const float* sbb = sb + static_cast<int64_t>(nb / p.block_rows_b) * p.lds_b;
    const float* sx[NT][2];
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = min(tile.m0 + 8 * t + row_of(2 * q + i), tile.m1 - 1);
        sx[t][i] = p.sa + static_cast<int64_t>(m) * p.lds_a;
      }
    }
    // the scales of this warp's blocks of a stage, loaded a stage ahead
    BlockScales<NT> now[L::kBlocks], next[L::kBlocks];
    auto load_scales = [&](BlockScales<NT>(&v)[L::kBlocks], int ks) {
#pragma unroll
      for (int j = 0; j < L::kBlocks; ++j) {
        const int b = min(ks * L::kStageBlocks + j * L::kSlices + slice, blocks - 1);
        v[j].a = __ldg(sba + b);
        v[j].b = __ldg(sbb + b);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) v[j].x[t][i] = __ldg(sx[t][i] + b);
      }
    };
    if (p.k_stages > 0) load_scales(next, 0);
    for (int ks = 0; ks < p.k_stages; ++ks) {
#pragma unroll
      for (int j = 0; j < L::kBlocks; ++j) now[j] = next[j];
      load_scales(next, ks + 1);
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_abortable(&full_bar[stage], phase, p.timeout_ns,
                                                         p.status, abort_flag));
        if (!ok) *abort_flag = 1;
      }
      if (ok) {
#pragma unroll
        for (int j = 0; j < L::kBlocks; ++j) {
          const int in_stage = j * L::kSlices + slice;
          // (TMA fills zeros past K in a block it loads)
          if (ks * L::kStageBlocks + in_stage >= blocks) break;
          const uint8_t* w = smem + stage * L::kStage + in_stage * L::kBlockBytes;
          const uint8_t* x = w + (L::kRowsW + gr) * kBlock;
          w += (group * 16 + gr) * kBlock;
          uint4 wa[2], wb[2];
          int piece[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            piece[h] = ((4 * h + q) ^ gr) << 4;
            wa[h] = *reinterpret_cast<const uint4*>(w + piece[h]);
            wb[h] = *reinterpret_cast<const uint4*>(w + 8 * kBlock + piece[h]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 v = *reinterpret_cast<const uint4*>(x + 8 * t * kBlock + piece[h]);
              mma_e4m3(c, wa[h].x, wb[h].x, wa[h].y, wb[h].y, v.x, v.y);
              mma_e4m3(c, wa[h].z, wb[h].z, wa[h].w, wb[h].w, v.z, v.w);
            }
            acc[t][0] = fmaf(c[0], now[j].x[t][0] * now[j].a, acc[t][0]);
            acc[t][1] = fmaf(c[1], now[j].x[t][1] * now[j].a, acc[t][1]);
            acc[t][2] = fmaf(c[2], now[j].x[t][0] * now[j].b, acc[t][2]);
            acc[t][3] = fmaf(c[3], now[j].x[t][1] * now[j].b, acc[t][3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_bar[stage]);
      }
      if (++stage == L::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (L::kSlices > 1) {
      // Two buffers: slice 0 has read a buffer when it comes to the barrier of
      // the next tile, which the others pass before they write it again.  (A
      // warp that gave up still comes to every barrier.)
      float* mine = red + (turn * kMmaWarps + warp) * NT * 4 * 32 + lane;
      turn ^= 1;
      if (slice != 0) {
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) mine[i * 32] = acc[i / 4][i % 4];
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (slice != 0) continue;
      for (int v = 1; v < L::kSlices; ++v)
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) acc[i / 4][i % 4] += mine[(v * RG * NT * 4 + i) * 32];
    }
    if (!ok) continue;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = tile.m0 + 8 * t + row_of(2 * q + (i & 1));
        const int n = tile.n0 + group * 16 + gr + 8 * (i >> 1);
        if (m >= tile.m1 || n >= p.N) continue;
        const int64_t at = m * p.ldd + n;
        float v = p.alpha * acc[t][i];
        if (p.beta != 0.0f) v = fmaf(p.beta, load_as_f32(p.D, at, p.dtype_d), v);
        if (p.flags & kEpiBias)
          v += load_as_f32(p.bias, tile.expert * p.stride_bias + n, p.dtype_d);
        if (p.flags & kEpiGelu) v = gelu2(make_float2(v, v)).x;
        if (p.dtype_d == DG_F32)
          static_cast<float*>(p.D)[at] = v;
        else
          static_cast<uint16_t*>(p.D)[at] = static_cast<uint16_t>(
              p.dtype_d == DG_BF16 ? BF16::pack(v, 0.0f) : F16::pack(v, 0.0f));
      }
  }
}

template <int NT, int RG>
cudaError_t run_skinny(const Fp8Args& a, SkinnyParams p) {
  using L = SkinnySmem<NT, RG>;
  p.tiles_n = static_cast<int>((a.N + 16 * RG - 1) / (16 * RG));
  p.most_blocks = static_cast<uint32_t>(kMaxTiles / p.tiles_n);
  const int64_t stage_k = L::kStageBlocks * kBlock;
  p.k_stages = static_cast<int>((a.K + stage_k - 1) / stage_k);
  CUtensorMap ta{}, tb{};
  cudaError_t e = cudaSuccess;
  if (a.K > 0) {
    const int64_t pitch = p.offsets ? a.stride_b / a.ldb : 0;
    p.b_rows = static_cast<int>(pitch);
    const int64_t b_rows = p.offsets ? (a.count - 1) * pitch + a.N : a.N;
    e = tc::encode_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, a.M, a.K, a.lda, L::kRowsX,
                          kBlock, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    e = tc::encode_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, b_rows, a.K, a.ldb, L::kRowsW,
                          kBlock, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  auto kern = skinny_fp8_kernel<NT, RG>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  e = once_per_device(attr_set, dev, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::bytes(kMaxExperts));
  });
  if (e != cudaSuccess) return e;
  const int64_t chunks = p.offsets ? a.M / (8 * NT) + std::min(a.count, a.M)
                                   : (a.M + 8 * NT - 1) / (8 * NT);
  if (chunks * p.tiles_n > kMaxTiles) return cudaErrorInvalidConfiguration;
  const int64_t ctas = std::min<int64_t>(chunks * p.tiles_n, a.sm_count);
  e = launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads),
                       static_cast<size_t>(L::bytes(p.offsets ? a.count : 0)), a.stream, ta, tb, p);
  count_launches(1);
  return e;
}

template <int NT>
cudaError_t run_rows(const Fp8Args& a, const SkinnyParams& p) {
  const int64_t products =
      p.offsets ? std::min(a.count, a.M) : (a.M + 8 * NT - 1) / (8 * NT);
  // (1 x 8960 x 1536, 140 tiles of 64 rows on 152 SMs: 4.2 us, with tiles of 32
  // 5.5; 16 x 8192 x 8192, 128 tiles of 64: 16.7 us, of 32 18.6)
  if (2 * products * ((a.N + 63) / 64) >= a.sm_count) return run_skinny<NT, 4>(a, p);
  if (2 * products * ((a.N + 31) / 32) >= a.sm_count) return run_skinny<NT, 2>(a, p);
  return run_skinny<NT, 1>(a, p);
}

}  // namespace

cudaError_t launch_fp8_skinny(const Fp8Args& a) {
  SkinnyParams p;
  p.sa = a.sa;
  p.lds_a = a.lds_a;
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
  p.count = p.offsets ? static_cast<int>(a.count) : 0;
  p.flags = a.epi;
  p.dtype_d = static_cast<int>(a.dtype_d);
  p.block_rows_b = a.block_rows_b;
  p.tiles_n = p.k_stages = p.b_rows = 0;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  const int64_t rows_each = p.offsets ? (a.M + a.count - 1) / a.count : a.M;
  if (rows_each <= 8) return run_rows<1>(a, p);
  if (rows_each <= 16) return run_rows<2>(a, p);
  return run_rows<4>(a, p);
}

}  // namespace dg
