// A whole mixture-of-experts layer for a few tokens (dg_moe_layer in dg.h) in
// two kernels:
//   up:    h[s] = act(W1[e] x_t + b1[e])    for each slot s = (t, j), e = ids[s]
//   down:  y[t] = sum over j of weights[t,j] (W2[e] h[s] + b2[e])
//
// The job is to read the used experts' weights once, at the rate of HBM: 8-bit
// codes (FP8) or 4-bit codes and their scales (NVF4).  Both kernels are the same
// machine: a persistent CTA per SM takes units (32 weight rows of one expert, up
// to 8 of its slots), one thread keeps a ring of TMA loads in flight across
// units, and 8 warps multiply with warp-level E4M3 MMAs (m16n8k32, weights as the
// 16-row operand).
//
// Activations stay exact: a value times a power of two is split into three E4M3
// parts, p0 = e4m3(v), p1 = e4m3(16 (v - p0)), p2 = e4m3(16 (16 (v - p0) - p1)),
// v = p0 + p1 / 16 + p2 / 256.  Each part carries 4 bits and a sign, so 16-bit
// inputs are represented exactly down to 2^-25 of their row's largest value, and
// h, FP32 before, with an error of at most 2^-13 of each value or 2^-25 of the
// largest of 32.  The parts are columns of the MMA of their own, and with a slot
// or two per expert they cost nothing: the 8 columns are there anyway.
//
// 4-bit codes become E4M3 by two shifts and masks per four codes (e2m1 = 64
// times the E4M3 value with the same bits) and keep their order in memory, so 32
// values of an MMA lie in two blocks with a scale each.  Each part therefore
// takes two columns, one for each block, with zeros in the other block's place.
//
// Units that end in the same outputs meet in fixed order: slots' sums go to
// scratch, and whichever warp finishes the last slot of a token (counted by
// atomics that the results do not depend on) adds them in the order of j.
#include <algorithm>

#include "epilogue.cuh"
#include "fp8.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kMmaWarps = 8;
constexpr int kThreads = (kMmaWarps + 1) * 32;
constexpr int kTileRows = 32;  // weight rows per unit (twice as many where gated)
constexpr int kMaxChunk = 8;   // slots per unit

enum : int { kFp8 = 0, kNvf4 = 1 };

struct LayerParams {
  const int32_t* ids;
  int tokens, top_k, slots, count, chunk;
  // the phase's product: K values (k_blocks of 128 bytes), `rows` results
  int K, k_blocks, k_tiles, rows, tiles, up0;
  int w_rows, sf_rows;       // weight rows, scale tile rows from one expert to the next
  const float* sw;           // FP8 block scales
  int64_t lds_w, stride_sw;
  const float* row_w;        // NVF4 row scales
  int64_t stride_row;
  const void* bias;
  int64_t stride_bias;
  int bf16;                  // X, D and the biases
  const uint16_t* X;
  int64_t ldx;
  int x_pitch;               // bytes of a row of parts in shared memory
  uint8_t* h;                // parts of h, 3 rows per slot in sorted order, ldh bytes each
  int64_t ldh;
  float* hs;                 // their scales, one per 32 values, hs_ld per slot
  int hs_ld;
  float* part;               // slots' sums of the second product
  unsigned* done;            // [tiles][tokens]: slots finished
  int done_words;
  const float* weights;
  uint16_t* D;
  int64_t ldd;
  int stages, act_boxes, block_bytes;
  int off_x, off_red, off_route;
  int* status;
  uint64_t timeout_ns;
};

// The routing in shared memory: slots sorted by expert (stable), cut into
// chunks of at most `chunk` slots of one expert.
struct Route {
  int *pos, *slot;         // slot -> sorted place (-1: dropped), and back
  int *expert, *first, *n; // per chunk
  int *valid;              // per token: its slots that are not dropped
  float* fx;               // per token: what its parts are multiplied by
  unsigned* amax;          // per token
  int* ids;
  int *cnt, *start, *base; // per expert
  int* chunks;             // their number
};
__device__ __forceinline__ Route route_at(int* m, const LayerParams& p) {
  Route r;
  r.ids = m;
  r.pos = r.ids + (p.slots + 3) / 4 * 4;
  r.slot = r.pos + p.slots;
  r.expert = r.slot + p.slots;
  r.first = r.expert + p.slots;
  r.n = r.first + p.slots;
  r.valid = r.n + p.slots;
  r.fx = reinterpret_cast<float*>(r.valid + p.tokens);
  r.amax = reinterpret_cast<unsigned*>(r.fx + p.tokens);
  r.cnt = reinterpret_cast<int*>(r.amax + p.tokens);
  r.start = r.cnt + p.count;
  r.base = r.start + p.count;
  r.chunks = r.base + p.count;
  return r;
}
int route_bytes(int64_t slots, int64_t tokens, int64_t count) {
  return static_cast<int>(4 * ((slots + 3) / 4 * 4 + 5 * slots + 3 * tokens + 3 * count + 4));
}

// All threads of the CTA; ends with a barrier.
__device__ __forceinline__ void build_route(const Route& r, const LayerParams& p) {
  for (int e = threadIdx.x; e < p.count; e += kThreads) r.cnt[e] = 0;
  for (int t = threadIdx.x; t < p.tokens; t += kThreads) r.valid[t] = 0, r.amax[t] = 0u;
  for (int s = threadIdx.x; s < (p.slots + 3) / 4 * 4; s += kThreads) {
    const int e = s < p.slots ? __ldg(p.ids + s) : -1;
    r.ids[s] = e >= 0 && e < p.count ? e : -1;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.slots; s += kThreads) {
    const int e = r.ids[s];
    int rank = -1;
    if (e >= 0) {
      rank = 0;  // slots of this expert before s
      const int4* v = reinterpret_cast<const int4*>(r.ids);
      for (int i = 0; i <= s / 4; ++i) {
        const int4 w = v[i];
        rank += (4 * i < s && w.x == e) + (4 * i + 1 < s && w.y == e) + (4 * i + 2 < s && w.z == e) +
                (4 * i + 3 < s && w.w == e);
      }
      atomicAdd(&r.cnt[e], 1);  // counts: the order does not matter
      atomicAdd(&r.valid[s / p.top_k], 1);
    }
    r.pos[s] = rank;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0, run_c = 0;
    for (int e0 = 0; e0 < p.count; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < p.count ? r.cnt[e] : 0, k = (c + p.chunk - 1) / p.chunk;
      int v = c, w = k;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v, d), b = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) v += a, w += b;
      }
      if (e < p.count) r.start[e] = run + v - c, r.base[e] = run_c + w - k;
      run += __shfl_sync(0xffffffffu, v, 31);
      run_c += __shfl_sync(0xffffffffu, w, 31);
    }
    if (lane == 0) *r.chunks = run_c;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.slots; s += kThreads)
    if (r.ids[s] >= 0) {
      const int at = r.start[r.ids[s]] + r.pos[s];
      r.pos[s] = at;
      r.slot[at] = s;
    }
  for (int e = threadIdx.x; e < p.count; e += kThreads) {
    const int c = r.cnt[e];
    for (int i = 0, k = r.base[e]; i < c; i += p.chunk, ++k) {
      r.expert[k] = e;
      r.first[k] = r.start[e] + i;
      r.n[k] = min(p.chunk, c - i);
    }
  }
  __syncthreads();
}

// The power of two f with amax f in (224, 448], as its inverse; 1 for zero.
__device__ __forceinline__ float parts_factor(float amax, float& inverse) {
  const uint32_t b = __float_as_uint(amax);
  // 448 = 1.75 * 2^8
  int e = 127 + 8 - static_cast<int>(b >> 23) - ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = min(max(e, -120), 120);
  if (amax == 0.0f) e = 0;
  inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return F16::unpack(h);
}
// Four scaled values -> their three parts, four codes each.
__device__ __forceinline__ void split4(float (&v)[4], uint32_t (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    part[i] = e4m3x4(v[0], v[1], v[2], v[3]);
    if (i == 2) break;
    const float2 a = e4m3x2_values(part[i] & 0xFFFFu), b = e4m3x2_values(part[i] >> 16);
    v[0] = 16.0f * (v[0] - a.x), v[1] = 16.0f * (v[1] - a.y);
    v[2] = 16.0f * (v[2] - b.x), v[3] = 16.0f * (v[3] - b.y);
  }
}

// Eight 16-bit values of a row of K from k on, zeros past its end.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int K) {
  if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0u;
    const uint32_t hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The tokens' parts in shared memory, three rows per token; 4-bit weights'
// order: of each 32 values the even ones, then the odd ones.  A token with an
// infinity or a NaN has parts of zeros and the factor NaN.
template <int Fmt, typename T>
__device__ __forceinline__ void load_tokens(const LayerParams& p, uint8_t* parts, const Route& r) {
  const int padded = p.k_blocks * (Fmt == kFp8 ? 128 : 256);
  const int per_row = (padded + 255) / 256 * 32;  // pieces of 8 values: whole warps
  const int pieces = p.tokens * per_row;
  for (int i = threadIdx.x; i < pieces; i += kMmaWarps * 32) {
    const int t = i / per_row, k = (i - t * per_row) * 8;
    const uint4 v = load8(p.X + t * p.ldx, k, p.K);
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                          __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if ((threadIdx.x & 31) == 0) atomicMax(&r.amax[t], m);
  }
  asm volatile("bar.sync 1, 256;" ::: "memory");
  for (int i = threadIdx.x; i < pieces; i += kMmaWarps * 32) {
    const int t = i / per_row, k = (i - t * per_row) * 8;
    const unsigned bits = r.amax[t];
    const bool odd = bits >= T::kInf;
    float inv;
    const float f = parts_factor(T::one(odd ? 0u : bits), inv);
    if (k == 0) r.fx[t] = odd ? CUDART_NAN_F : inv;
    const uint4 v = odd ? make_uint4(0u, 0u, 0u, 0u) : load8(p.X + t * p.ldx, k, p.K);
    const float2 a = T::unpack(v.x), b = T::unpack(v.y), c = T::unpack(v.z), d = T::unpack(v.w);
    if (k >= padded) continue;
    uint8_t* row = parts + t * 3 * p.x_pitch;
    uint32_t lo[3], hi[3];
    if (Fmt == kFp8) {
      float x[4] = {a.x * f, a.y * f, b.x * f, b.y * f}, y[4] = {c.x * f, c.y * f, d.x * f, d.y * f};
      split4(x, lo);
      split4(y, hi);
#pragma unroll
      for (int i3 = 0; i3 < 3; ++i3)
        *reinterpret_cast<uint2*>(row + i3 * p.x_pitch + k) = make_uint2(lo[i3], hi[i3]);
    } else {
      float x[4] = {a.x * f, b.x * f, c.x * f, d.x * f}, y[4] = {a.y * f, b.y * f, c.y * f, d.y * f};
      split4(x, lo);
      split4(y, hi);
      const int at = (k & ~31) + (k & 31) / 2;
#pragma unroll
      for (int i3 = 0; i3 < 3; ++i3) {
        *reinterpret_cast<uint32_t*>(row + i3 * p.x_pitch + at) = lo[i3];
        *reinterpret_cast<uint32_t*>(row + i3 * p.x_pitch + at + 16) = hi[i3];
      }
    }
  }
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a (16 x 32, weights) . b (32 x 8, activations)
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The low (high) nibbles of four bytes of E2M1 codes as E4M3 codes of 1/64 of
// their values: sign to bit 7, exponent and mantissa to bits 4 .. 2.
__device__ __forceinline__ uint32_t e4m3_of_low(uint32_t w) {
  return ((w << 4) & 0x80808080u) | ((w << 2) & 0x1C1C1C1Cu);
}
__device__ __forceinline__ uint32_t e4m3_of_high(uint32_t w) {
  return (w & 0x80808080u) | ((w >> 2) & 0x1C1C1C1Cu);
}

__device__ __forceinline__ float as_f32(const void* p, int64_t i, int bf16) {
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return bf16 ? BF16::one(h) : F16::one(h);
}
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269504f;
  return __fdividef(g, 1.0f + ex2_approx(-kLog2e * g));
}

// Down: the second product (its activations come with the ring's stages).  NT:
// tiles of 8 columns that a unit can have.
template <int Fmt, bool Down, bool Gated, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_sf,
                     const __grid_constant__ CUtensorMap tmap_h,
                     const __grid_constant__ LayerParams p) {
  static_assert(!(Down && Gated), "the second product has no gate");
  constexpr int RG = Gated ? 4 : 2;        // groups of 16 rows
  constexpr int kSlices = kMmaWarps / RG;  // warps that share a group's K blocks
  constexpr int kBlockW = 16 * RG * 128;
  constexpr int kBlockS = Fmt == kNvf4 ? RG / 2 * 2048 : 0;
  constexpr int kAcc = Fmt == kFp8 ? 4 : 2;         // sums per lane and column tile
  constexpr int kPerTile = Fmt == kFp8 ? 8 : 4;     // parts per column tile
  constexpr int kActHalves = Fmt == kFp8 ? 1 : 2;   // 128-byte pieces of a block's activations

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stage_bytes = kSlices * p.block_bytes;
  uint8_t* xparts = smem + p.off_x;
  float* red = reinterpret_cast<float*>(smem + p.off_red);  // [2][warp][NT * kAcc][lane]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(red + 2 * kMmaWarps * NT * kAcc * 32);
  uint64_t* empty_bar = full_bar + p.stages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty_bar + p.stages);
  const Route r = route_at(reinterpret_cast<int*>(smem + p.off_route), p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kMmaWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarps && lane == 0) {
    tma_prefetch_desc(&tmap_w);
    if (Fmt == kNvf4) tma_prefetch_desc(&tmap_sf);
    if (Down) tma_prefetch_desc(&tmap_h);
  }
  // The second kernel starts while the first one runs: what it reads before it
  // waits (choices and weights) was there before the first, which waited for
  // every kernel before it ahead of letting this one start.
  if (!Down) grid_dependency_wait();
  build_route(r, p);
  const int chunks = *r.chunks;
  const int units = chunks * p.tiles;
  const int k_stages = (p.k_blocks + kSlices - 1) / kSlices;

  if (warp == kMmaWarps) {
    // ------------------------------------------------------------ producer
    if (!elect_one_lane()) return;
    const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
    int64_t issued = 0;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // the loads of K stage ks of unit t: weights, or activations
    auto load = [&](int t, int ks, int st, bool weights, bool acts) {
      const int tile = t / chunks, u = t - tile * chunks;
      const int e = r.expert[u];
      const int b0 = ks * kSlices, n = min(kSlices, p.k_blocks - b0);
      const int boxes = Down ? (3 * r.n[u] + 7) / 8 : 0;
      uint8_t* dst = smem + st * stage_bytes;
      if (weights)
        mbar_arrive_expect_tx(&full_bar[st], static_cast<uint32_t>(
                                                 n * (kBlockW + kBlockS + boxes * kActHalves * 1024)));
      for (int j = 0; j < n; ++j, dst += p.block_bytes) {
        const int kb = b0 + j;
        if (weights) {
          const int row = e * p.w_rows + tile * kTileRows;
          tma_load_2d(&tmap_w, &full_bar[st], dst, kb * 128, row, stream);
          if (Gated)
            tma_load_2d(&tmap_w, &full_bar[st], dst + kBlockW / 2, kb * 128, row + p.up0, stream);
          if (Fmt == kNvf4) {
            const int sf = (e * p.sf_rows + (tile >> 2)) * p.k_tiles + 4 * kb;
            tma_load_2d(&tmap_sf, &full_bar[st], dst + kBlockW, 0, sf, keep);
            if (Gated)
              tma_load_2d(&tmap_sf, &full_bar[st], dst + kBlockW + 2048, 0,
                          sf + (p.up0 >> 7) * p.k_tiles, keep);
          }
        }
        if (Down && acts)
          for (int b = 0; b < boxes; ++b)
#pragma unroll
            for (int h = 0; h < kActHalves; ++h)
              tma_load_2d(&tmap_h, &full_bar[st],
                          dst + kBlockW + kBlockS + (b * kActHalves + h) * 1024,
                          (kb * kActHalves + h) * 128, 3 * r.first[u] + 8 * b, keep);
      }
    };
    int64_t ahead = 0;
    if (Down) {
      // the first stages' weights before the first kernel has finished
      int st = 0;
      for (int t = blockIdx.x; t < units && st < p.stages; t += gridDim.x)
        for (int ks = 0; ks < k_stages && st < p.stages; ++ks, ++st) load(t, ks, st, true, false);
      ahead = st;
      grid_dependency_wait();
      st = 0;
      for (int t = blockIdx.x; t < units && st < ahead; t += gridDim.x)
        for (int ks = 0; ks < k_stages && st < ahead; ++ks, ++st) load(t, ks, st, false, true);
    }
    for (int t = blockIdx.x; t < units && ok; t += gridDim.x)
      for (int ks = 0; ks < k_stages; ++ks) {
        if (issued >= ahead) {
          ok = mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status,
                                   abort_flag);
          if (!ok) break;
          load(t, ks, stage, true, true);
        }
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    grid_launch_dependents();
    if (!ok) *abort_flag = 1;
    // the copies land before the CTA goes away, whoever gave up
    const int64_t first = issued > p.stages ? issued - p.stages : 0;
    for (int64_t i = first; i < issued; ++i)
      mbar_wait(&full_bar[i % p.stages], static_cast<uint32_t>((i / p.stages) & 1), p.timeout_ns,
                p.status);
    return;
  }

  // ------------------------------------------------------------------- MMAs
  if (Down) {
    grid_dependency_wait();
    // tokens without an expert
    for (int t = 0; t < p.tokens; ++t)
      if (r.valid[t] == 0)
        for (int n = blockIdx.x * 256 + threadIdx.x; n < p.rows; n += gridDim.x * 256)
          p.D[t * p.ldd + n] = 0;
  } else {
    for (int i = blockIdx.x * 256 + threadIdx.x; i < p.done_words; i += gridDim.x * 256)
      p.done[i] = 0u;
    if (p.bf16)
      load_tokens<Fmt, BF16>(p, xparts, r);
    else
      load_tokens<Fmt, F16>(p, xparts, r);
  }
  const int g = lane >> 2, q = lane & 3;
  const int group = warp % RG, slice = warp / RG;
  // ldmatrix: lanes 8 i .. 8 i + 7 give the rows of matrix i
  const int mat = lane >> 3, mrow = lane & 7;
  // weights: matrices (rows 0-7, piece), (rows 8-15, piece), and of the next piece
  const int a_row = mrow + 8 * (mat & 1);
  const uint32_t a_base = static_cast<uint32_t>((group * 16 + a_row) * 128);
  const uint32_t a_swz = static_cast<uint32_t>(a_row & 7);
  const uint32_t b_mask = (q >> 1) == (g & 1) ? 0xffffffffu : 0u;  // NVF4: the column's block
  const uint32_t smem0 = smem_addr(smem);
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int t = blockIdx.x; t < units; t += gridDim.x) {
    const int tile = t / chunks, u = t - tile * chunks;
    const int e = r.expert[u], n = r.n[u], first = r.first[u];
    const int cols = (3 * n + kPerTile - 1) / kPerTile;  // column tiles in use
    float acc[NT][kAcc];
    uint32_t b_base[NT];   // this lane's row of activations for ldmatrix
    const float* hs[NT][2];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
#pragma unroll
      for (int i = 0; i < kAcc; ++i) acc[c][i] = 0.0f;
      // the part of this lane's column (past the last: the last's)
      const int part = min(c * kPerTile + (Fmt == kFp8 ? mrow : mrow >> 1), 3 * n - 1);
      if (!Down)
        b_base[c] = smem_addr(xparts) +
                    static_cast<uint32_t>((r.slot[first + part / 3] / p.top_k * 3 + part % 3) * p.x_pitch);
      else
        b_base[c] = static_cast<uint32_t>((part >> 3) * kActHalves * 1024 + (part & 7) * 128);
      if (Down)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int mine = min(c * kPerTile + (Fmt == kFp8 ? 2 * q + i : q), 3 * n - 1);
          hs[c][i] = p.hs + static_cast<int64_t>(first + mine / 3) * p.hs_ld;
        }
    }
    // FP8: the scales of this lane's rows' weight blocks
    const float *swa = nullptr, *swb = nullptr;
    if (Fmt == kFp8) {
      const int row = (Gated && group >= 2 ? p.up0 - 32 : 0) + tile * kTileRows + group * 16 + g;
      const int last = p.rows - 1 + (Gated && group >= 2 ? p.up0 : 0);
      const float* sw = p.sw + e * p.stride_sw;
      swa = sw + static_cast<int64_t>(min(row, last) / 128) * p.lds_w;
      swb = sw + static_cast<int64_t>(min(row + 8, last) / 128) * p.lds_w;
    }
    // the block's scales (of weights, and of h), loaded a stage ahead
    float sa = 0.0f, sb = 0.0f, sa_next = 0.0f, sb_next = 0.0f;
    float hv[NT][2][Fmt == kFp8 ? 4 : 8], hv_next[NT][2][Fmt == kFp8 ? 4 : 8];
    auto load_scales = [&](int kb) {
      kb = min(kb, p.k_blocks - 1);
      if (Fmt == kFp8) {
        sa_next = __ldg(swa + kb);
        sb_next = __ldg(swb + kb);
      }
      if (Down)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (c >= cols) break;
#pragma unroll
          for (int i = 0; i < (Fmt == kFp8 ? 2 : 1); ++i)
#pragma unroll
            for (int k = 0; k < (Fmt == kFp8 ? 1 : 2); ++k) {
              const float4 v =
                  *reinterpret_cast<const float4*>(hs[c][i] + kb * (Fmt == kFp8 ? 4 : 8) + 4 * k);
              hv_next[c][i][4 * k] = v.x, hv_next[c][i][4 * k + 1] = v.y;
              hv_next[c][i][4 * k + 2] = v.z, hv_next[c][i][4 * k + 3] = v.w;
            }
        }
    };
    load_scales(slice);
    for (int ks = 0; ks < k_stages; ++ks) {
      sa = sa_next, sb = sb_next;
      if (Down)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < (Fmt == kFp8 ? 4 : 8); ++k) hv[c][i][k] = hv_next[c][i][k];
      const int kb = ks * kSlices + slice;
      load_scales(kb + kSlices);
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_abortable(&full_bar[stage], phase, p.timeout_ns,
                                                         p.status, abort_flag));
        if (!ok) *abort_flag = 1;
      }
      if (ok && kb < p.k_blocks) {
        const uint32_t block = smem0 + static_cast<uint32_t>(stage * stage_bytes + slice * p.block_bytes);
        const uint32_t acts = block + kBlockW + kBlockS;
        if (Fmt == kFp8) {
          float c4[NT][4];
          uint32_t b[NT][4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a[4];
            ldmatrix4(a, block + a_base + (((2 * m + (mat >> 1)) ^ a_swz) << 4));
#pragma unroll
            for (int c = 0; c < NT; ++c) {
              if (c >= cols) break;
              if (m % 2 == 0) {
                // pieces 2 m .. 2 m + 3: two MMAs' worth
                const uint32_t piece = static_cast<uint32_t>(2 * m + mat);
                ldmatrix4(b[c], Down ? acts + b_base[c] + ((piece ^ ((b_base[c] >> 7) & 7)) << 4)
                                     : b_base[c] + static_cast<uint32_t>(kb * 128) + (piece << 4));
              }
              if (Down || m == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) c4[c][i] = 0.0f;
              mma_e4m3(c4[c], a[0], a[1], a[2], a[3], b[c][2 * (m & 1)], b[c][2 * (m & 1) + 1]);
              if (Down) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  acc[c][i] = fmaf(c4[c][i], (i < 2 ? sa : sb) * hv[c][i & 1][m], acc[c][i]);
              } else if (m == 3) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][i] = fmaf(c4[c][i], i < 2 ? sa : sb, acc[c][i]);
              }
            }
          }
        } else {
          // this lane's scale words: rows g and g + 8 of the group, four blocks each
          const int line = (group & 1) * 16 + g;
          const uint32_t sf = block + kBlockW + (group >> 1) * 2048 +
                              static_cast<uint32_t>(line * 16 + (tile & 3) * 4);
#pragma unroll
          for (int mm = 0; mm < 4; ++mm) {
            if (4 * kb + mm >= p.k_tiles) break;  // (a scale tile past the last is another's)
            uint32_t w[4], sg, sh;
            ldmatrix4(w, block + a_base + (((2 * mm + (mat >> 1)) ^ a_swz) << 4));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sg) : "r"(sf + mm * 512));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sh) : "r"(sf + mm * 512 + 128));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float2 s0 = e4m3x2_values((sg >> (16 * half)) & 0xFFFFu);
              const float2 s1 = e4m3x2_values((sh >> (16 * half)) & 0xFFFFu);
              const uint32_t a0 = e4m3_of_low(w[2 * half]), a2 = e4m3_of_high(w[2 * half]);
              const uint32_t a1 = e4m3_of_low(w[2 * half + 1]), a3 = e4m3_of_high(w[2 * half + 1]);
#pragma unroll
              for (int c = 0; c < NT; ++c) {
                if (c >= cols) break;
                uint32_t b[2];
                // 32 values of a part: pieces 4 mm + 2 half (even ones) and the next (odd)
                const uint32_t piece = static_cast<uint32_t>(4 * mm + 2 * half + (mat & 1));
                const uint32_t at =
                    Down ? acts + b_base[c] + (piece >> 3) * 1024 +
                               (((piece & 7) ^ ((b_base[c] >> 7) & 7)) << 4)
                         : b_base[c] + static_cast<uint32_t>(kb * 256) + (piece << 4);
                asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                             : "=r"(b[0]), "=r"(b[1])
                             : "r"(at)
                             : "memory");
                float c4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_e4m3(c4, a0, a1, a2, a3, b[0] & b_mask, b[1] & b_mask);
                const float t0 = fmaf(c4[1], s0.y, c4[0] * s0.x);
                const float t1 = fmaf(c4[3], s1.y, c4[2] * s1.x);
                if (Down) {
                  acc[c][0] = fmaf(t0, hv[c][0][2 * mm + half], acc[c][0]);
                  acc[c][1] = fmaf(t1, hv[c][0][2 * mm + half], acc[c][1]);
                } else {
                  acc[c][0] += t0;
                  acc[c][1] += t1;
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&empty_bar[stage]);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // The slices' sums meet in shared memory.  Two buffers: every warp has read
    // one when it comes to the barrier of the next unit, which the others pass
    // before they write it again.  (A warp that gave up still comes there.)
    float* mine = red + (turn * kMmaWarps + warp) * NT * kAcc * 32 + lane;
    const float* all = red + turn * kMmaWarps * NT * kAcc * 32;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NT * kAcc; ++i)
      if (i / kAcc < cols) mine[i * 32] = acc[i / kAcc][i % kAcc];
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (!ok || warp >= n) continue;
    // warp: slot of the unit; lane: row of the tile
    auto total = [&](int rows_group) {
      float v = 0.0f;
#pragma unroll
      for (int i = 2; i >= 0; --i) {
        const int part = 3 * warp + i;
        const int c = part / kPerTile, in = part % kPerTile;
        // the lane and register that hold row `lane` of the tile
        const int who = Fmt == kFp8 ? (lane & 7) * 4 + in / 2 : (lane & 7) * 4 + in;
        const int reg = Fmt == kFp8 ? (in & 1) + 2 * ((lane >> 3) & 1) : (lane >> 3) & 1;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k)
          s += all[((k * RG + rows_group + (lane >> 4)) * NT * kAcc + c * kAcc + reg) * 32 + who];
        v = fmaf(v, 0.0625f, s);
      }
      return v;
    };
    const int row = tile * kTileRows + lane;
    const int pos = first + warp, slot = r.slot[pos], token = slot / p.top_k;
    const bool there = row < p.rows;
    // what the code's bits stand for beside their E4M3 value, and the row's scale
    auto scaled = [&](float v, int of_row) {
      if (Fmt == kNvf4) v *= 64.0f * (there ? __ldg(p.row_w + e * p.stride_row + of_row) : 0.0f);
      if (!Down) v *= r.fx[token];
      if (p.bias && there) v += as_f32(p.bias, e * p.stride_bias + of_row, p.bf16);
      return v;
    };
    if (!Down) {
      float v = scaled(total(0), row);
      if (Gated) {
        const float up = scaled(total(2), row + p.up0);
        v = silu(v) * up;
      } else {
        v = gelu2(make_float2(v, v)).x;
      }
      if (!there) v = 0.0f;
      const uint32_t bits = __float_as_uint(v) & 0x7FFFFFFFu;
      const uint32_t most = __reduce_max_sync(0xffffffffu, bits);
      const bool odd = most >= 0x7F800000u;
      float inv;
      const float f = parts_factor(__uint_as_float(odd ? 0u : most), inv);
      float x[4] = {odd ? 0.0f : v * f, 0.0f, 0.0f, 0.0f};
      uint32_t code[3];
      split4(x, code);
      const int at = Fmt == kFp8 ? lane : (lane & 1) * 16 + (lane >> 1);
      uint8_t* h = p.h + static_cast<int64_t>(3 * pos) * p.ldh + tile * kTileRows + at;
#pragma unroll
      for (int i = 0; i < 3; ++i) h[i * p.ldh] = static_cast<uint8_t>(code[i]);
      // (the last tile also fills what the second product reads past it)
      const int more = tile == p.tiles - 1 ? p.hs_ld - tile : 1;
      if (lane < more)
        p.hs[static_cast<int64_t>(pos) * p.hs_ld + tile + lane] =
            lane == 0 ? (odd ? CUDART_NAN_F : inv) : 0.0f;
    } else {
      float v = scaled(total(0), row);
      if (there) __stcg(p.part + static_cast<int64_t>(pos) * p.rows + row, v);
      __threadfence();
      __syncwarp();
      unsigned before = 0;
      if (lane == 0) before = atomicAdd(p.done + static_cast<int64_t>(tile) * p.tokens + token, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (static_cast<int>(before) != r.valid[token] - 1) continue;
      // the token's last slot: its slots in order
      __threadfence();
      if (!there) continue;
      float y = 0.0f;
      for (int j = 0; j < p.top_k; ++j) {
        const int at = r.pos[token * p.top_k + j];
        if (at < 0) continue;
        const float w = p.weights ? __ldg(p.weights + token * p.top_k + j) : 1.0f;
        y = fmaf(w, __ldcg(p.part + static_cast<int64_t>(at) * p.rows + row), y);
      }
      p.D[token * p.ldd + row] =
          static_cast<uint16_t>(p.bf16 ? BF16::pack(y, 0.0f) : F16::pack(y, 0.0f));
    }
  }
}

constexpr int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Where the scratch's parts lie.
struct LayerScratch {
  int64_t ldh, hs_ld, h, hs, part, done, bytes;
};
LayerScratch scratch_of(const MoeLayerArgs& a) {
  LayerScratch s;
  const int64_t slots = a.tokens * a.top_k;
  s.ldh = round_up(a.hidden, 256);
  s.hs_ld = s.ldh / 32;
  s.h = 0;
  s.hs = s.h + 3 * slots * s.ldh;
  s.part = s.hs + slots * s.hs_ld * 4;
  s.done = s.part + round_up(slots * a.out * 4, 16);
  s.bytes = s.done + round_up((a.out + kTileRows - 1) / kTileRows * a.tokens * 4, 16);
  return s;
}

// Shared memory besides the ring, and the ring's stages in `room` bytes.
template <int NT, int kAcc>
int red_bytes() {
  return 2 * kMmaWarps * NT * kAcc * 32 * 4;
}

template <int Fmt, bool Down, bool Gated, int NT>
cudaError_t run_phase(const MoeLayerArgs& a, LayerParams p, int x_bytes) {
  constexpr int RG = Gated ? 4 : 2, kSlices = kMmaWarps / RG, kAcc = Fmt == kFp8 ? 4 : 2;
  constexpr int kMaxSmem = 227 * 1024;
  const MoeWeights& w = Down ? a.down : a.up;
  const int64_t n_rows = Down ? a.out : a.hidden * (Gated ? 2 : 1);
  const int64_t bytes_k = Fmt == kFp8 ? p.K : (p.K + 1) / 2;
  p.k_blocks = static_cast<int>((bytes_k + 127) / 128);
  p.k_tiles = static_cast<int>((p.K + 63) / 64);
  p.tiles = (p.rows + kTileRows - 1) / kTileRows;
  const int64_t pitch = a.count > 1 ? w.stride / w.ld : n_rows;
  p.w_rows = static_cast<int>(pitch);
  p.sf_rows = static_cast<int>((n_rows + 127) / 128);
  p.sw = static_cast<const float*>(w.scales);
  p.lds_w = w.lds;
  p.stride_sw = w.stride_s;
  p.row_w = w.row_scales;
  p.stride_row = n_rows;
  p.bias = w.bias;
  p.stride_bias = w.stride_bias;
  p.act_boxes = Down ? (3 * p.chunk + 7) / 8 : 0;
  p.block_bytes = 16 * RG * 128 + (Fmt == kNvf4 ? RG / 2 * 2048 : 0) +
                  p.act_boxes * (Fmt == kNvf4 ? 2 : 1) * 1024;
  const int stage = kSlices * p.block_bytes;
  const int red = red_bytes<NT, kAcc>();
  const int route = route_bytes(p.slots, p.tokens, p.count);
  const int fixed = static_cast<int>(round_up(x_bytes, 16)) + red + 256 + route + 1024;
  // Two CTAs' worth of ring where the rest leaves room: the second kernel's
  // starts to fill while the first one's ends.
  int room = 112 * 1024 - fixed;
  if (room < 4 * stage) room = kMaxSmem - fixed;
  p.stages = std::min(8, room / stage);
  if (p.stages < 2) return cudaErrorInvalidValue;
  p.off_x = p.stages * stage;
  p.off_red = p.off_x + static_cast<int>(round_up(x_bytes, 16));
  p.off_route = p.off_red + red + 256;
  const int smem = p.off_route + route + 1024;

  CUtensorMap tw{}, ts{}, th{};
  cudaError_t e = tc::encode_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes,
                                    (a.count - 1) * pitch + n_rows, bytes_k, w.ld, kTileRows, 128,
                                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  ts = th = tw;  // not used by every variant
  if (Fmt == kNvf4) {
    e = tc::encode_map_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_UINT32, w.scales,
                          static_cast<int64_t>(p.sf_rows) * p.k_tiles * a.count, 128, 512, 4, 128,
                          CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  if (Down) {
    // what the first kernel writes: whole tiles of 32 values
    e = tc::encode_map_2d(&th, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.h, 3 * a.tokens * a.top_k,
                          round_up(a.hidden, kTileRows), p.ldh, 8, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  auto kern = moe_layer_kernel<Fmt, Down, Gated, NT>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  e = once_per_device(attr_set, dev, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t most = std::min<int64_t>(p.slots, int64_t(1) << 20) * p.tiles;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(most, a.sm_count));
  e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                       static_cast<size_t>(smem), a.stream, tw, ts, th, p);
  count_launches(1);
  return e;
}

template <int Fmt, int NT>
cudaError_t run_layer(const MoeLayerArgs& a, LayerParams p, int x_bytes) {
  p.K = static_cast<int>(a.width);
  p.rows = static_cast<int>(a.hidden);
  p.up0 = static_cast<int>(a.hidden);
  const cudaError_t e = a.gated ? run_phase<Fmt, false, true, NT>(a, p, x_bytes)
                                : run_phase<Fmt, false, false, NT>(a, p, x_bytes);
  if (e != cudaSuccess) return e;
  p.K = static_cast<int>(a.hidden);
  p.rows = static_cast<int>(a.out);
  return run_phase<Fmt, true, false, NT>(a, p, 0);
}

}  // namespace

int64_t moe_layer_scratch(const MoeLayerArgs& a) { return scratch_of(a).bytes; }

// Bytes of the tokens' parts in shared memory: rows of whole 256-value blocks,
// 16 bytes apart in their banks.
static int64_t parts_bytes(int64_t tokens, int64_t width) {
  return 3 * tokens * (round_up(width, 256) + 16);
}
// What is left of a CTA's shared memory beside a ring of two stages, its sums
// and the routing.
bool moe_layer_fits(const MoeLayerArgs& a) {
  const int64_t slots = a.tokens * a.top_k;
  return slots <= kMaxLayerSlots &&
         parts_bytes(a.tokens, a.width) + route_bytes(slots, a.tokens, a.count) <= 146 * 1024;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a) {
  const LayerScratch s = scratch_of(a);
  uint8_t* base = static_cast<uint8_t*>(a.scratch);
  LayerParams p{};
  p.ids = a.ids;
  p.tokens = static_cast<int>(a.tokens);
  p.top_k = static_cast<int>(a.top_k);
  p.slots = static_cast<int>(a.tokens * a.top_k);
  p.count = static_cast<int>(a.count);
  p.bf16 = a.bf16;
  p.X = static_cast<const uint16_t*>(a.X);
  p.ldx = a.ldx;
  p.x_pitch = static_cast<int>(round_up(a.width, 256)) + 16;
  p.h = base + s.h;
  p.ldh = s.ldh;
  p.hs = reinterpret_cast<float*>(base + s.hs);
  p.hs_ld = static_cast<int>(s.hs_ld);
  p.part = reinterpret_cast<float*>(base + s.part);
  p.done = reinterpret_cast<unsigned*>(base + s.done);
  p.done_words = static_cast<int>((a.out + kTileRows - 1) / kTileRows * a.tokens);
  p.weights = a.weights;
  p.D = static_cast<uint16_t*>(a.D);
  p.ldd = a.ldd;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  const int x_bytes = static_cast<int>(parts_bytes(a.tokens, a.width));
  // Slots per unit: as many as there are tokens can meet in one expert (a token
  // that names an expert twice gets a unit more), at most 8.
  const bool few = a.tokens <= 2;
  p.chunk = few ? 2 : kMaxChunk;
  if (a.nvf4) return few ? run_layer<kNvf4, 2>(a, p, x_bytes) : run_layer<kNvf4, 6>(a, p, x_bytes);
  return few ? run_layer<kFp8, 1>(a, p, x_bytes) : run_layer<kFp8, 3>(a, p, x_bytes);
}

}  // namespace dg
