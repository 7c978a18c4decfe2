// Expert routing: tokens' choices sorted by expert, rows moved into that
// order and back (weighted), and the way back's gradient.  dg.h states each
// operator; the quantizing way there is in fp8_quant.cu.
#include <algorithm>

#include <cuda_runtime.h>

#include "fp8.cuh"

namespace dg {
namespace {

using namespace fp8;

// ---------------------------------------------------------------------------
// Sort: a stable counting sort in one launch of one thread-block cluster
// ---------------------------------------------------------------------------
// The slots are cut into one contiguous run per CTA of the cluster and those
// into one run per warp, so that (CTA, warp, position) is slot order and the
// result is stable whatever the timing:
//   1. each warp counts its run by expert in its own row of counters;
//   2. per expert, the warps' counts become running sums; the CTAs exchange
//      their totals through distributed shared memory, and every CTA computes
//      the segments' starts;
//   3. each warp walks its run again, 32 slots at a time: lanes with the same
//      expert find each other with one ballot per bit of its number (a match
//      instruction takes longer: 131 thousand slots 31 us, with ballots 15) and
//      take the rows from the expert's running count on, in lane order.
// Bound by latency: the slots are read twice (8 bytes) and written once, a
// few hundred kilobytes at most (64 slots 3.3 us, 131 thousand 14.6).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxCtas = 8;  // the portable cluster size

struct SortParams {
  const int32_t* ids;
  int slots, count, align_mask;  // align - 1
  int per_warp;                  // slots per warp, a multiple of 32
  int warps;                     // per CTA that get slots
  int bits;                      // of an expert's number
  int64_t rows;
  int32_t *offsets, *row_slot, *slot_row;
};

__device__ __forceinline__ int ld_cluster_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The experts of slots s, s + 32, ...: -1 past `last` and where the choice is
// dropped.  All loads are under way before the first is used.
constexpr int kSortAhead = 8;
__device__ __forceinline__ void load_experts(const SortParams& p, int s, int last,
                                             int (&e)[kSortAhead]) {
#pragma unroll
  for (int i = 0; i < kSortAhead; ++i) e[i] = s + 32 * i < last ? __ldg(p.ids + s + 32 * i) : -1;
#pragma unroll
  for (int i = 0; i < kSortAhead; ++i)
    if (e[i] >= p.count) e[i] = -1;
#pragma unroll
  for (int i = 0; i < kSortAhead; ++i) e[i] = max(e[i], -1);
}

// The lanes whose expert is this lane's (-1 is no expert's number: its bits are
// those of the last, its sign sets it apart).
__device__ __forceinline__ unsigned same_lanes(int e, int bits) {
  unsigned m = __ballot_sync(0xffffffffu, e < 0);
  m = e < 0 ? m : ~m;
  for (int b = 0; b < bits; ++b) {
    const unsigned set = __ballot_sync(0xffffffffu, (e >> b) & 1);
    m &= (e >> b) & 1 ? set : ~set;
  }
  return m;
}

__global__ void __launch_bounds__(kSortThreads)
    moe_sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int sort_smem[];
  const int count = p.count;
  int* totals = sort_smem;                // [count]: this CTA's slots per expert
  int* start = totals + count;            // [count]: first row of this CTA's slots
  int* seg = start + count;               // [count]: slots per expert over all CTAs
  int* offs = seg + count;                // [count + 1]
  int* hist = offs + count + 1;           // [kSortWarps][count]
  __shared__ int warp_sum[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  for (int i = threadIdx.x; i < p.warps * count; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  grid_dependency_wait();

  const int64_t first64 = (static_cast<int64_t>(rank) * p.warps + warp) * p.per_warp;
  const int first = static_cast<int>(warp < p.warps && first64 < p.slots ? first64 : p.slots);
  const int64_t last64 = first64 + p.per_warp;
  const int last = static_cast<int>(last64 < p.slots ? last64 : p.slots);
  int* mine = hist + warp * count;
  for (int s0 = first; s0 < last; s0 += 32 * kSortAhead) {
    int e[kSortAhead];
    load_experts(p, s0 + lane, last, e);
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      if (s0 + 32 * i >= last) break;
      if (e[i] >= 0) atomicAdd(&mine[e[i]], 1);  // a count: the order does not matter
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < count; e += kSortThreads) {
    int sum = 0;
    for (int w0 = 0; w0 < p.warps; w0 += 8) {
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = w0 + i < p.warps ? hist[(w0 + i) * count + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (w0 + i < p.warps) hist[(w0 + i) * count + e] = sum;
        sum += c[i];
      }
    }
    totals[e] = sum;
  }
  __syncthreads();
  cluster_sync();  // every CTA's totals are there (a barrier of one CTA's threads without peers)
  // count <= kSortThreads: one expert per thread
  int before = 0, all = 0;
  if (threadIdx.x < count) {
    const uint32_t a = smem_addr(totals + threadIdx.x);
    for (int r = 0; r < ctas; ++r) {
      const int v = ld_cluster_int(mapa_shared(a, static_cast<uint32_t>(r)));
      if (r < rank) before += v;
      all += v;
    }
  }
  const int padded = (all + p.align_mask) & ~p.align_mask;
  int incl = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  if (threadIdx.x < count) {
    const int end = incl + (warp > 0 ? warp_sum[warp - 1] : 0);
    offs[threadIdx.x + 1] = end;
    start[threadIdx.x] = end - padded + before;
    seg[threadIdx.x] = all;
    if (threadIdx.x == 0) offs[0] = 0;
    if (rank == 0) {
      p.offsets[threadIdx.x + 1] = end;
      if (threadIdx.x == 0) p.offsets[0] = 0;
    }
  }
  // the peers have read this CTA's totals before it leaves
  cluster_arrive_release();
  __syncthreads();

  for (int s0 = first; s0 < last; s0 += 32 * kSortAhead) {
    int e[kSortAhead];
    load_experts(p, s0 + lane, last, e);
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      const int s = s0 + 32 * i + lane;
      if (s0 + 32 * i >= last) break;
      const unsigned same = same_lanes(e[i], p.bits);
      const unsigned below = same & ((1u << lane) - 1u);
      int row = -1;
      if (e[i] >= 0) row = start[e[i]] + mine[e[i]] + __popc(below);
      __syncwarp();
      if (e[i] >= 0 && below == 0) mine[e[i]] += __popc(same);
      __syncwarp();
      if (s < last) {
        p.slot_row[s] = row;
        if (row >= 0) p.row_slot[row] = s;
      }
    }
  }
  // -1 in the padding of each segment and past the last one
  if (p.align_mask != 0) {
    for (int e = rank * kSortWarps + warp; e < count; e += ctas * kSortWarps)
      for (int r = offs[e] + seg[e] + lane; r < offs[e + 1]; r += 32) p.row_slot[r] = -1;
  }
  const int64_t all_threads = static_cast<int64_t>(ctas) * kSortThreads;
  for (int64_t r = offs[count] + rank * kSortThreads + threadIdx.x; r < p.rows; r += all_threads)
    p.row_slot[r] = -1;
  cluster_wait_acquire();
}

// ---------------------------------------------------------------------------
// Rows there and back
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

// Eight 16-bit values from p, of which the first n (1 .. 8) exist.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n) {
  if (n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < n ? p[2 * i] : 0u;
    const uint32_t hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Rows are written once and read by a later kernel: a streaming store leaves
// L2 to the rows that are read again (4096 tokens to 16384 rows of 2048: 21.8
// us, 27.4 with plain stores).
__device__ __forceinline__ void store8(uint16_t* p, const uint4& v, int n) {
  if (n >= 8) {
    __stcs(reinterpret_cast<uint4*>(p), v);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = T::unpack(w[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(T::pack(f[0], f[1]), T::pack(f[2], f[3]), T::pack(f[4], f[5]),
                    T::pack(f[6], f[7]));
}

struct RowsParams {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* Y;
  int64_t ldy;
  uint16_t* D;
  int64_t ldd;
  const int32_t *row_slot, *slot_row;
  const float* weights;
  float* dweights;
  int64_t tokens, rows;
  int top_k, width, chunks;  // chunks of 8 values per row
  int64_t row_blocks;        // combine_backward: CTAs past the tokens' that clear padding rows
};

// D[r] = X[row_slot[r] / top_k], zeros without a slot: a warp per row.  Bound by
// the stores (16384 tokens of 2048 to 139 thousand rows: 130 us, 4390 GB/s
// written; 4096 tokens to 16384 rows, about L2's size: 21.8 us).
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
       r < p.rows; r += step) {
    const int slot = __ldg(p.row_slot + r);
    const int t = slot < 0 ? -1 : static_cast<int>(static_cast<unsigned>(slot) / p.top_k);
    const uint16_t* src = t >= 0 && t < p.tokens ? p.X + t * p.ldx : nullptr;
    uint16_t* dst = p.D + r * p.ldd;
#pragma unroll 4
    for (int c = lane; c < p.chunks; c += 32) {
      const int n = p.width - 8 * c;
      store8(dst + 8 * c, src ? load8(src + 8 * c, n) : make_uint4(0u, 0u, 0u, 0u), n);
    }
  }
}

// codes[r], scales[r] = those of X's row row_slot[r] / top_k (codes 0 and the
// scale of an empty block without a slot): a warp per row.  Bound by the stores
// (16384 tokens of 2048 to 139 thousand rows: 77 us with the tokens'
// quantization, 3820 GB/s written; clearing a buffer reaches 4060).
struct CodesParams {
  const uint8_t* X;  // codes of the tokens, pitch ldx bytes, a multiple of 16
  int64_t ldx;
  const float* sx;  // [tokens][blocks]
  uint8_t* D;
  int64_t ldd;
  float* sd;
  int64_t lds;
  const int32_t* row_slot;
  int64_t tokens, rows;
  int top_k, width, blocks;
};

__global__ void __launch_bounds__(kRowThreads)
    dispatch_codes_kernel(const __grid_constant__ CodesParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
       r < p.rows; r += step) {
    const int slot = __ldg(p.row_slot + r);
    const int t = slot < 0 ? -1 : static_cast<int>(static_cast<unsigned>(slot) / p.top_k);
    const bool there = t >= 0 && t < p.tokens;
    const uint8_t* src = p.X + (there ? t * p.ldx : 0);
    uint8_t* dst = p.D + r * p.ldd;
#pragma unroll 4
    for (int k = lane * 16; k < p.width; k += 512) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (there) v = *reinterpret_cast<const uint4*>(src + k);  // written by the kernel before
      if (k + 16 <= p.width) {
        __stcs(reinterpret_cast<uint4*>(dst + k), v);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (k + i < p.width) dst[k + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
      }
    }
    for (int b = lane; b < p.blocks; b += 32)
      p.sd[r * p.lds + b] =
          there ? p.sx[static_cast<int64_t>(t) * p.blocks + b] : __fdiv_rn(kFloor, kTop);
  }
}

// D[t] = sum over j of weights[t, j] * Y[slot_row[t, j]]: a thread takes eight
// columns of one token and loads kInFlight of its rows at a time; FP32 sums
// in the order of j.  Bound by memory: the rows are read once (8192 tokens of
// 4096 in 8 rows each, this and the gradient below: 374 us, 6470 GB/s; 8
// tokens 2.6 us).
constexpr int kInFlight = 8;

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t t = i / p.chunks;
  const int c = static_cast<int>(i - t * p.chunks);
  if (t >= p.tokens) return;
  const int n = p.width - 8 * c;
  float sum[8] = {};
  const int64_t s0 = t * p.top_k;
  for (int j0 = 0; j0 < p.top_k; j0 += kInFlight) {
    uint4 v[kInFlight];
    float w[kInFlight];
    bool there[kInFlight];
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      const int r = j0 + j < p.top_k ? __ldg(p.slot_row + s0 + j0 + j) : -1;
      there[j] = r >= 0 && r < p.rows;
      w[j] = there[j] && p.weights ? __ldg(p.weights + s0 + j0 + j) : 1.0f;
      if (there[j]) v[j] = load8(p.Y + r * p.ldy + 8 * c, n);
    }
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      if (!there[j]) continue;
      float y[8];
      unpack8<T>(v[j], y);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] = fmaf(w[j], y[q], sum[q]);
    }
  }
  store8(p.D + t * p.ldd + 8 * c, pack8<T>(sum), n);
}

// The way back's gradient.  CTA t < tokens: dY[slot_row[t, j]] = weights[t, j]
// * dD[t] and dweights[t, j] = dD[t] . Y[slot_row[t, j]], kInFlight slots at
// a time, dD[t] read once per such batch.  Later CTAs clear the padding rows.
// Bound by memory for wide rows (8192 tokens in 8 rows each, width 4096: 192 us,
// 6300 GB/s); narrow ones leave threads of a CTA without work (width 1024 88 us,
// 3430 GB/s; 256 47 us, 1640).
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ float part[kRowThreads / 32][kInFlight];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= p.tokens) {
    constexpr int kWarps = kRowThreads / 32;
    for (int64_t r = (blockIdx.x - p.tokens) * kWarps + warp; r < p.rows;
         r += p.row_blocks * kWarps) {
      if (__ldg(p.row_slot + r) >= 0) continue;
      for (int c = lane; c < p.chunks; c += 32)
        store8(p.D + r * p.ldd + 8 * c, make_uint4(0u, 0u, 0u, 0u), p.width - 8 * c);
    }
    return;
  }
  const int64_t t = blockIdx.x;
  const int64_t s0 = t * p.top_k;
  for (int j0 = 0; j0 < p.top_k; j0 += kInFlight) {
    int row[kInFlight];
    float w[kInFlight], dot[kInFlight];
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      const int r = j0 + j < p.top_k ? __ldg(p.slot_row + s0 + j0 + j) : -1;
      row[j] = r < p.rows ? r : -1;
      w[j] = row[j] >= 0 && p.weights ? __ldg(p.weights + s0 + j0 + j) : 1.0f;
      dot[j] = 0.0f;
    }
    for (int c = threadIdx.x; c < p.chunks; c += kRowThreads) {
      const int n = p.width - 8 * c;
      float d[8];
      unpack8<T>(load8(p.X + t * p.ldx + 8 * c, n), d);
      uint4 v[kInFlight];
      if (p.dweights) {
#pragma unroll
        for (int j = 0; j < kInFlight; ++j)
          if (row[j] >= 0) v[j] = load8(p.Y + row[j] * p.ldy + 8 * c, n);
      }
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        if (row[j] < 0) continue;
        float y[8];
        if (p.dweights) {
          unpack8<T>(v[j], y);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot[j] = fmaf(d[q], y[q], dot[j]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = w[j] * d[q];
        store8(p.D + row[j] * p.ldd + 8 * c, pack8<T>(y), n);
      }
    }
    if (!p.dweights) continue;
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kInFlight && j0 + threadIdx.x < p.top_k) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < kRowThreads / 32; ++v) sum += part[v][threadIdx.x];
      p.dweights[s0 + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

RowsParams rows_params(const MoeRowsJob& j) {
  RowsParams p;
  p.X = static_cast<const uint16_t*>(j.X);
  p.ldx = j.ldx;
  p.Y = static_cast<const uint16_t*>(j.Y);
  p.ldy = j.ldy;
  p.D = static_cast<uint16_t*>(j.D);
  p.ldd = j.ldd;
  p.row_slot = j.row_slot;
  p.slot_row = j.slot_row;
  p.weights = j.weights;
  p.dweights = j.dweights;
  p.tokens = j.tokens;
  p.rows = j.rows;
  p.top_k = static_cast<int>(j.top_k);
  p.width = static_cast<int>(j.width);
  p.chunks = static_cast<int>((j.width + 7) / 8);
  p.row_blocks = 0;
  return p;
}

int64_t sort_smem_bytes(int64_t count) { return ((4 + kSortWarps) * count + 1) * 4; }

}  // namespace

cudaError_t launch_moe_sort(const MoeSortJob& j, cudaStream_t stream) {
  SortParams p;
  p.ids = j.ids;
  p.slots = static_cast<int>(j.tokens * j.top_k);
  p.count = static_cast<int>(j.count);
  p.align_mask = static_cast<int>(j.align - 1);
  p.rows = j.rows;
  p.offsets = j.offsets;
  p.row_slot = j.row_slot;
  p.slot_row = j.slot_row;
  // one CTA for each 2048 slots (64 per warp), up to the cluster's eight; a
  // warp takes at least 32
  const int64_t want = (static_cast<int64_t>(p.slots) + 2047) / 2048;
  int ctas = 1;
  while (ctas < kSortMaxCtas && ctas < want) ctas *= 2;
  const int64_t per_cta = (static_cast<int64_t>(p.slots) + ctas - 1) / ctas;
  const int64_t steps = ((per_cta + kSortWarps - 1) / kSortWarps + 31) / 32;
  const int64_t per_warp = std::max<int64_t>(1, steps) * 32;
  p.per_warp = static_cast<int>(per_warp);
  p.bits = 0;
  while ((1 << p.bits) < j.count) ++p.bits;
  p.warps = static_cast<int>(std::max<int64_t>(1, (per_cta + per_warp - 1) / per_warp));

  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = once_per_device(attr_set, dev, [&]() {
    return cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sort_smem_bytes(kMaxExperts)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(sort_smem_bytes(j.count));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, moe_sort_kernel, p);
  count_launches(1);
  return e;
}

cudaError_t launch_moe_dispatch(const MoeRowsJob& j, cudaStream_t stream, int sm_count) {
  const RowsParams p = rows_params(j);
  const int64_t ctas = (j.rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t cap = static_cast<int64_t>(sm_count) * 8 * 4;
  const cudaError_t e =
      launch_dependent(dispatch_kernel, dim3(static_cast<unsigned>(std::min(ctas, cap))),
                       dim3(kRowThreads), 0, stream, p);
  count_launches(1);
  return e;
}

cudaError_t launch_moe_dispatch_codes(const Fp8RowsJob& j, const void* codes, int64_t ldx,
                                      const float* scales, cudaStream_t stream, int sm_count) {
  CodesParams p;
  p.X = static_cast<const uint8_t*>(codes);
  p.ldx = ldx;
  p.sx = scales;
  p.D = static_cast<uint8_t*>(j.codes);
  p.ldd = j.ldq;
  p.sd = j.scales;
  p.lds = j.lds;
  p.row_slot = j.row_slot;
  p.tokens = j.tokens;
  p.rows = j.rows;
  p.top_k = static_cast<int>(j.top_k);
  p.width = static_cast<int>(j.K);
  p.blocks = static_cast<int>((j.K + kBlock - 1) / kBlock);
  const int64_t ctas = (j.rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t cap = static_cast<int64_t>(sm_count) * 8 * 4;
  const cudaError_t e =
      launch_dependent(dispatch_codes_kernel, dim3(static_cast<unsigned>(std::min(ctas, cap))),
                       dim3(kRowThreads), 0, stream, p);
  count_launches(1);
  return e;
}

cudaError_t launch_moe_combine(const MoeRowsJob& j, cudaStream_t stream) {
  const RowsParams p = rows_params(j);
  const int64_t ctas = (j.tokens * p.chunks + kRowThreads - 1) / kRowThreads;
  const dim3 grid(static_cast<unsigned>(ctas));
  const cudaError_t e =
      j.bf16 ? launch_dependent(combine_kernel<BF16>, grid, dim3(kRowThreads), 0, stream, p)
             : launch_dependent(combine_kernel<F16>, grid, dim3(kRowThreads), 0, stream, p);
  count_launches(1);
  return e;
}

cudaError_t launch_moe_combine_backward(const MoeRowsJob& j, cudaStream_t stream) {
  RowsParams p = rows_params(j);
  // one CTA for each 64 rows looks for padding (8 rows per warp)
  p.row_blocks = (j.rows + 63) / 64;
  const dim3 grid(static_cast<unsigned>(j.tokens + p.row_blocks));
  const cudaError_t e =
      j.bf16
          ? launch_dependent(combine_backward_kernel<BF16>, grid, dim3(kRowThreads), 0, stream, p)
          : launch_dependent(combine_backward_kernel<F16>, grid, dim3(kRowThreads), 0, stream, p);
  count_launches(1);
  return e;
}

}  // namespace dg
