// A whole mixture-of-experts layer for a few tokens (dg_moe_layer in dg.h) in
// three kernels:
//   up:    h[s] = act(W1[e] x_t + b1[e])    for each slot s = (t, j), e = ids[s]
//   down:  z[s] = W2[e] h[s] + b2[e]
//   sum:   y[t] = sum over j of weights[t,j] z[t,j]
//
// The job is to read the used experts' weights once, at the rate of HBM: 8-bit
// codes (FP8) or 4-bit codes and their scales (NVF4).  Up and down are the same
// machine: a persistent CTA per SM takes units (32 weight rows of one expert, up
// to 8 of its slots, 4 in down), one thread keeps a ring of loads in flight across units, 8
// warps multiply with warp-level FP16 MMAs (m16n8k16, weights as the 16-row
// operand, slots as the 8 columns), and 3 warps take the units' sums in turn and
// finish them.
//
// Codes become FP16 exactly (an E4M3 value; an E2M1 value times its block's E4M3
// scale, 6 significant bits) by the pair conversions.  (E4M3 MMAs, which take FP8
// codes as they are, want the activations in three parts, and 4-bit codes' two
// blocks in columns of their own: 1340 clocks a stage of NVF4 against the 780 that
// HBM needs for it.)  Activations are FP16 times a power of two: x exactly, h
// as two FP16 values (22 bits) in two of the MMA's columns, each 32 of its values with
// a power of their own, so that h has FP32's range.  (With 11 bits its rounding is as
// large as that of an FP16 result; 16 tokens NVF4 72.8 us then, as units of the second
// product held eight slots.)
//
// What a lane needs for 32 values of K is then 16 bytes: in a 16-byte piece of a
// weight row as ldmatrix hands it out, lane q of a row's four has 4 (FP8) or 8
// (NVF4) codes, and the order of K inside an MMA is free as long as both operands
// share it.  FP8's 32 values are two pieces, so activations are stored with 4 of
// the one beside 4 of the other.
//
// h lies in scratch as the second kernel reads it: by K stage, then slot in
// sorted order, so that one bulk copy brings a unit's slots of a stage, values
// and scales.  Few copies matter: a TMA copy costs the issuing thread about 80
// clocks (with one for each K block and 8 rows, 990 clocks a stage).
//
// Measured, experts of 2048 x 2048, SwiGLU: 8 tokens, FP8, 454 MB of weights in 77
// us (5.9 TB/s; 6.2 and 5.7 in the two products by themselves: HBM); 16 tokens, NVF4, 335
// MB in 76.5 us (4.4 TB/s; 5.1 and 3.6: instructions, and h's two columns in the second).
// One token, 8 experts of 4096 x 2048, GELU: FP8 27.5 us, NVF4 22.6, of which the
// kernels' starts are 6.
#include <algorithm>

#include "convert.cuh"
#include "epilogue.cuh"
#include "fp8.cuh"
#include "tc_common.cuh"

namespace dg {
namespace {

using namespace fp8;

constexpr int kTeamWarps = 8;  // that share a stage
constexpr int kEpiWarps = 3;
constexpr int kTileRows = 32;  // weight rows per unit (twice as many where gated)
constexpr int kMaxChunk = 8;   // slots per unit
constexpr int kMaxChunkH = 4;  // in the second product: two columns each
constexpr int kMaxStages = 8;
constexpr int64_t kNextBytes = 48 * 1024;  // a CTA's part of what goes to L2 ahead

enum : int { kFp8 = 0, kNvf4 = 1 };

// What differs between the kernels: row groups of 16, the warps that share a
// group's K blocks (the blocks of a stage), values in a K block (128 bytes of each
// weight row), bytes of a stage's weights and of their scales.
//
// A team of 8 warps takes whole stages.  What hides a stage's latencies (a chain
// of loads, conversions and MMAs of 600 to 1200 clocks, where HBM brings a stage
// in 700 to 780) is a second team: two CTAs of one on an SM, where half its shared
// memory holds a ring, or two in a CTA, which take turns (8 tokens gated FP8: 82
// us, with one team 117).
template <int Fmt, bool Down, bool Gated, int Teams = 1>
struct Shape {
  static constexpr int kMmaWarps = Teams * kTeamWarps;
  static constexpr int kTmaWarp = kMmaWarps, kEpiWarp = kMmaWarps + 1;
  static constexpr int kThreads = (kMmaWarps + 1 + kEpiWarps) * 32;
  static constexpr int RG = Gated ? 4 : 2;
  static constexpr int kSlices = kTeamWarps / RG;
  static constexpr int kBlockK = Fmt == kFp8 ? 128 : 256;
  static constexpr int kBlockW = kTileRows * 128;
  static constexpr int kW = (Gated ? 2 : 1) * kSlices * kBlockW;
  static constexpr int kS = Fmt == kNvf4 ? (Gated ? 2 : 1) * kSlices * 2048 : 0;
  static constexpr int kRed = kEpiWarps * kMmaWarps * 4 * 32 * 4;
  static constexpr int kBars = (2 * kMaxStages + 2 * kEpiWarps + 1) * 8 + 8;
};
// A slot's share of a stage of the second product: FP16 values, what is left of
// them as FP16, then a scale for each 32 of them.  Rows are 64 bytes apart in their
// banks: two rows' 64-byte reads do not meet.
template <int Fmt>
struct HRow {
  static constexpr int kK =
      Shape<Fmt, true, false>::kSlices * Shape<Fmt, true, false>::kBlockK;
  static constexpr int kRest = 2 * kK, kScales = 4 * kK;
  static constexpr int kBytes = kScales + kK / 32 * 4 + (Fmt == kNvf4 ? 64 : 0);
  static_assert(kBytes % 128 == 64, "banks");
};

struct LayerParams {
  const int32_t* ids;
  int tokens, top_k, slots, count, chunk;
  int inv_chunk, inv_top_k;  // 2^16 / chunk, 2^20 / top_k, rounded up: for quotients of up to 519
  // the phase's product: K values (k_blocks of 128 bytes, full_blocks of them whole,
  // k_tiles scale tiles), `rows` results
  int K, k_blocks, full_blocks, k_tiles, rows, tiles, up0;
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
  int x_pitch;               // bytes of a token in shared memory
  uint8_t* h;                // [K stage][slot][HRow]
  float* part;               // slots' sums of the second product, part_pitch apart
  int64_t part_pitch;
  // the first kernel's: the weights of the second, to bring into L2
  const uint8_t* next_w;
  int64_t next_ld, next_stride;
  const uint8_t* next_sf;
  int64_t next_sf_stride;    // bytes from one expert's scale tiles to the next's
  int next_bytes, next_rows, next_k_tiles;
  int stages, stage_bytes;
  int off_x, off_red, off_route;
  int* status;
  uint64_t timeout_ns;
};

// The routing in shared memory: slots sorted by expert (stable), cut into
// chunks of at most `chunk` slots of one expert.
struct Route {
  int* of;                   // sorted place -> token, or slot
  int *expert, *first, *n;   // per chunk
  float* fx;                 // per token: what its values are multiplied by
  int *ids, *rank;           // per slot: expert; place among that expert's (-1: dropped)
  int *cnt, *seen, *start;   // per expert: its slots, twice; those of the experts before
  int* chunks;               // their number
};
__device__ __forceinline__ Route route_at(int* m, const LayerParams& p) {
  Route r;
  r.ids = m;
  r.rank = r.ids + p.slots;
  r.of = r.rank + p.slots;
  r.expert = r.of + p.slots;
  r.first = r.expert + p.slots;
  r.n = r.first + p.slots;
  r.fx = reinterpret_cast<float*>(r.n + p.slots);
  r.cnt = reinterpret_cast<int*>(r.fx + p.tokens);
  r.seen = r.cnt + p.count;
  r.start = r.seen + p.count;
  r.chunks = r.start + p.count;
  return r;
}
int route_bytes(int64_t slots, int64_t tokens, int64_t count) {
  return static_cast<int>(4 * (6 * slots + tokens + 3 * count + 1));
}

// The routing is built by the warp that loads: only who multiplies and finishes sums
// waits at a barrier for it.  What takes the time is the fetches of code that is in no
// cache yet, so it is short, without a division.  (The first kernel wants sorted places'
// tokens, the second their slots.)
//
// Up to 32 slots: a slot per lane (in the form below one token of 8 choices took 0.4 us
// longer in each product).
template <bool Down>
__device__ __forceinline__ void build_route_32(const Route& r, const LayerParams& p, int lane) {
  int e = lane < p.slots ? __ldg(p.ids + lane) : -1;
  if (e >= p.count) e = -1;
  int less = 0, same = 0, before = 0;  // slots of smaller experts, of this one, and of those before
  for (int j = 0; j < p.slots; ++j) {
    const int f = __shfl_sync(0xffffffffu, e, j);
    less += f >= 0 && f < e;
    same += f == e;
    before += f == e && j < lane;
  }
  const bool there = e >= 0;
  const int at = there ? less + before : -1;
  const bool starts = there && (before * p.inv_chunk >> 16) * p.chunk == before;
  const unsigned all = __ballot_sync(0xffffffffu, starts);
  int k = 0;  // chunks before this slot's
  for (int j = 0; j < p.slots; ++j) {
    const int f = __shfl_sync(0xffffffffu, at, j);
    k += (all >> j & 1u) && f < at;
  }
  if (there) r.of[at] = Down ? lane : lane * p.inv_top_k >> 20;
  if (starts) {
    r.expert[k] = e;
    r.first[k] = at;
    r.n[k] = min(p.chunk, same - before);
  }
  if (lane == 0) *r.chunks = __popc(all);
  __syncwarp();
}

// More: the warp that loads counts the experts' slots and cuts them into chunks, and
// goes on; another puts the slots in their places, 32 at a time.  A slot's rank is the
// number of its expert's slots in the blocks before and in the lanes below.
__device__ __forceinline__ void count_route(const Route& r, const LayerParams& p, int lane) {
#pragma unroll 1
  for (int e = lane; e < p.count; e += 32) r.cnt[e] = 0;
  __syncwarp();
#pragma unroll 4
  for (int s = lane; s < p.slots; s += 32) {
    const int e = __ldg(p.ids + s);
    if (e >= 0 && e < p.count) atomicAdd(&r.cnt[e], 1);  // counts: the order does not matter
  }
  __syncwarp();
  int run = 0;  // slots and (<< 16) chunks of the experts before, at most 512 each
#pragma unroll 1
  for (int e0 = 0; e0 < p.count; e0 += 32) {
    const int e = e0 + lane;
    const int c = e < p.count ? r.cnt[e] : 0;
    const int own = c | ((c + p.chunk - 1) * p.inv_chunk >> 16) << 16;
    int v = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += a;
    }
    int at = (run + v - own) & 0xFFFF, u = (run + v - own) >> 16;
    if (e < p.count) r.start[e] = at;
#pragma unroll 1
    for (int left = c; left > 0; left -= p.chunk, at += p.chunk, ++u) {
      r.expert[u] = e;
      r.first[u] = at;
      r.n[u] = min(p.chunk, left);
    }
    run += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) *r.chunks = run >> 16;
  __syncwarp();
  asm volatile("bar.arrive 2, 64;" ::: "memory");
}
template <bool Down>
__device__ __forceinline__ void place_route(const Route& r, const LayerParams& p, int lane) {
#pragma unroll 4
  for (int s = lane; s < p.slots; s += 32) r.ids[s] = __ldg(p.ids + s);
#pragma unroll 1
  for (int e = lane; e < p.count; e += 32) r.seen[e] = 0;
  __syncwarp();
#pragma unroll 1
  for (int s0 = 0; s0 < p.slots; s0 += 32) {
    const int s = s0 + lane;
    int e = s < p.slots ? r.ids[s] : -1;
    if (e >= p.count) e = -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int below = __popc(same & ((1u << lane) - 1u));
    const int before = e >= 0 ? r.seen[e] : 0;
    __syncwarp();
    if (e >= 0 && below == 0) r.seen[e] = before + __popc(same);
    if (s < p.slots) r.rank[s] = e >= 0 ? before + below : -1;
    __syncwarp();
  }
  asm volatile("bar.sync 2, 64;" ::: "memory");
#pragma unroll 1
  for (int s = lane; s < p.slots; s += 32)
    if (r.rank[s] >= 0) r.of[r.start[r.ids[s]] + r.rank[s]] = Down ? s : s * p.inv_top_k >> 20;
}

// A CTA's units, chunk by chunk of a tile (neighbours share a tile's place in
// different experts, or the weights).
struct UnitWalk {
  int tile, u, chunks, d_tile, d_u;
  __device__ __forceinline__ void start(int first, int step, int chunks_) {
    chunks = max(chunks_, 1);
    // (exact below 2^21: the quotient of a + 1/2 is half a chunk's part off an integer)
    tile = static_cast<int>(__fdividef(first + 0.5f, chunks));
    u = first - tile * chunks;
    d_tile = static_cast<int>(__fdividef(step + 0.5f, chunks));
    d_u = step - d_tile * chunks;
  }
  __device__ __forceinline__ void next() {
    tile += d_tile;
    u += d_u;
    if (u >= chunks) {
      u -= chunks;
      ++tile;
    }
  }
};

// The power of two that brings amax into [2^14, 2^15), and its inverse; 1 for
// zero.
__device__ __forceinline__ float half_factor(float amax, float& inverse) {
  int e = 127 + 14 - static_cast<int>(__float_as_uint(amax) >> 23);
  e = amax == 0.0f ? 0 : min(max(e, -120), 120);
  inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Where value k of 32 lies: NVF4's in order, FP8's 4 of the first 16 beside 4 of
// the second.
template <int Fmt>
__device__ __forceinline__ int place_of(int k) {
  return Fmt == kNvf4 ? k : (k & 12) << 1 | (k & 16) >> 2 | (k & 3);
}

// The largest finite magnitude of two bfloat16 values, as bits.
__device__ __forceinline__ uint32_t finite_max(uint32_t w) {
  const uint32_t a = w & 0x7FFFu, b = w >> 16 & 0x7FFFu;
  return max(a < BF16::kInf ? a : 0u, b < BF16::kInf ? b : 0u);
}
__device__ __forceinline__ uint32_t scaled_half2(uint32_t w, float f) {
  const float2 v = BF16::unpack(w);
  return F16::pack(v.x * f, v.y * f);
}

// The tokens in shared memory as FP16: FP16 as it is, BF16 times a power of two
// per token that brings its largest finite value near the top (infinities and
// NaNs stay what they are).  Bulk copies bring them (all CTAs want all of them: by
// loads into registers 16 tokens of 2048 took 9.5 us); an MMA warp per token then
// converts it in place.
__device__ __forceinline__ void copy_tokens(const LayerParams& p, uint8_t* xs, uint64_t* bar) {
  const uint32_t bytes = static_cast<uint32_t>(p.K / 8 * 16);
  if (bytes == 0) return;
  const uint64_t keep = policy_evict_last();
  mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.tokens) * bytes);
  for (int t = 0; t < p.tokens; ++t)
    bulk_load_g2s(xs + t * p.x_pitch, p.X + t * p.ldx, bytes, bar, keep);
}
template <int Fmt, int kWarps>
__device__ __forceinline__ bool convert_tokens(const LayerParams& p, uint8_t* xs, const Route& r,
                                               uint64_t* bar, int warp, int lane) {
  const int padded = p.k_blocks * Shape<Fmt, false, false>::kBlockK, whole = p.K / 8 * 8;
  // what the bulk copies leave: the last values, and zeros past them
  for (int t = warp; t < p.tokens; t += kWarps)
    for (int k = whole + lane; k < padded; k += 32)
      reinterpret_cast<uint16_t*>(xs + t * p.x_pitch)[k] = k < p.K ? p.X[t * p.ldx + k] : 0;
  if (whole > 0 && !__all_sync(0xffffffffu, mbar_wait(bar, 0, p.timeout_ns, p.status))) return false;
  __syncwarp();
  for (int t = warp; t < p.tokens; t += kWarps) {
    uint8_t* row = xs + t * p.x_pitch;
    float f = 1.0f, inv = 1.0f;
    if (p.bf16) {
      uint32_t m = 0;
      for (int k = lane * 8; k < padded; k += 256) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + k * 2);
        m = max(max(m, max(finite_max(v.x), finite_max(v.y))),
                max(finite_max(v.z), finite_max(v.w)));
      }
      f = half_factor(BF16::one(__reduce_max_sync(0xffffffffu, m)), inv);
    }
    if (lane == 0) r.fx[t] = inv;
    if (Fmt == kNvf4) {
      if (p.bf16)
        for (int k = lane * 8; k < padded; k += 256) {
          uint4* at = reinterpret_cast<uint4*>(row + k * 2);
          const uint4 v = *at;
          *at = make_uint4(scaled_half2(v.x, f), scaled_half2(v.y, f), scaled_half2(v.z, f),
                           scaled_half2(v.w, f));
        }
    } else {
      for (int k = lane * 32; k < padded; k += 1024) {
        uint4* at = reinterpret_cast<uint4*>(row + k * 2);
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = at[i];
          if (p.bf16)
            v[i] = make_uint4(scaled_half2(v[i].x, f), scaled_half2(v[i].y, f),
                              scaled_half2(v[i].z, f), scaled_half2(v[i].w, f));
        }
        // values 4 q .. 4 q + 3 beside 16 + 4 q ..
        at[0] = make_uint4(v[0].x, v[0].y, v[2].x, v[2].y);
        at[1] = make_uint4(v[0].z, v[0].w, v[2].z, v[2].w);
        at[2] = make_uint4(v[1].x, v[1].y, v[3].x, v[3].y);
        at[3] = make_uint4(v[1].z, v[1].w, v[3].z, v[3].w);
      }
    }
  }
  return true;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t ld_shared1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared1(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// c += a (16 x 16, weights) . b (16 x 8, activations)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 codes -> two FP16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The scales (E4M3 codes in bytes `at` and at + 2 of a word) as FP16 pairs of
// the same value.
__device__ __forceinline__ void scale_pairs(uint32_t word, uint32_t at, uint32_t (&s)[2]) {
  const uint32_t two = __byte_perm(word, 0u, 0x4420u + 0x0011u * at);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  // (a multiplication takes a half twice without an instruction of its own)
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "mov.b32 %0, {a, a};\n\t"
      "mov.b32 %1, {b, b};\n\t}"
      : "=r"(s[0]), "=r"(s[1])
      : "r"(h));
}

__device__ __forceinline__ float as_f32(const void* p, int64_t i, int bf16) {
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return bf16 ? BF16::one(h) : F16::one(h);
}
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269504f;
  return __fdividef(g, 1.0f + ex2_approx(-kLog2e * g));
}

// t * row * power + bias, one rounding: the power of two goes to the row's scale, or, where
// that leaves FP32's normal range, to t (NVF4's, between 2^-34 and 2^60 where it is not
// zero), which comes back into range with the row's scale if the result is in it.  (FP8 has
// no row scale, and a power alone is in range.)
__device__ __forceinline__ float scaled_sum(float t, float row, float power, float bias) {
  const float s = row * power;
  const bool in = (fabsf(s) >= 0x1p-126f && fabsf(s) <= 0x1.fffffep127f) || row == 0.0f;
  return fmaf(in ? t : t * power, in ? s : row, bias);
}

__device__ __forceinline__ void prefetch_l2(const uint8_t* at, uint32_t bytes) {
  if (bytes > 0)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
// Weights of the second product into L2, by the thread whose last loads have
// landed: HBM would wait for the second kernel until the first one's last sums are
// done and its own first loads are out.  (One token, FP8 27.7 us, was 29.2; with 128
// KB a CTA 29.0, for NVF4 later than without; before the last loads have landed 28.1.)
// They are the second kernel's first where its chunks and grid are the first one's: up
// to four slots an expert, as with one token.  Else they are others that it reads: it
// cuts an expert's slots by four, the first by eight.
template <int Fmt>
__device__ __forceinline__ void prefetch_next(const LayerParams& p, const Route& r, int chunks,
                                              int step) {
  const int tiles = (p.next_rows + kTileRows - 1) / kTileRows;
  int64_t left = kNextBytes;
  UnitWalk walk{};
  walk.start(blockIdx.x, step, chunks);
  for (; walk.tile < tiles && left > 0; walk.next()) {
    const int e = r.expert[walk.u], row = walk.tile * kTileRows;
    const int64_t bytes = (min(kTileRows, p.next_rows - row) - 1) * p.next_ld + p.next_bytes;
    prefetch_l2(p.next_w + e * p.next_stride + row * p.next_ld,
                static_cast<uint32_t>(min(bytes, left)) & ~15u);
    if (Fmt == kNvf4)  // a quarter of the tiles of 128 rows
      prefetch_l2(p.next_sf + e * p.next_sf_stride +
                      ((walk.tile >> 2) * 4 + (walk.tile & 3)) * static_cast<int64_t>(p.next_k_tiles) * 128,
                  static_cast<uint32_t>(p.next_k_tiles) * 128);
    left -= bytes;
  }
}

// Down: the second product (its activations come with the ring's stages).
template <int Fmt, bool Down, bool Gated, int Teams>
__global__ void __launch_bounds__(Shape<Fmt, Down, Gated, Teams>::kThreads, Teams == 1 ? 2 : 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_tail,
                     const __grid_constant__ CUtensorMap tmap_sf,
                     const __grid_constant__ LayerParams p) {
  static_assert(!(Down && Gated), "the second product has no gate");
  using S = Shape<Fmt, Down, Gated, Teams>;
  using H = HRow<Fmt>;
  constexpr int RG = S::RG, kSlices = S::kSlices, kMmaWarps = S::kMmaWarps;
  constexpr int kTmaWarp = S::kTmaWarp, kEpiWarp = S::kEpiWarp;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem + p.off_x;
  float* red = reinterpret_cast<float*>(smem + p.off_red);  // [kEpiWarps][warp][4][lane]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + p.off_red + S::kRed);
  uint64_t* empty_bar = full_bar + kMaxStages;
  uint64_t* red_full = empty_bar + kMaxStages;
  uint64_t* red_empty = red_full + kEpiWarps;
  uint64_t* x_bar = red_empty + kEpiWarps;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(x_bar + 1);
  const Route r = route_at(reinterpret_cast<int*>(smem + p.off_route), p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kTeamWarps);
    }
    for (int b = 0; b < kEpiWarps; ++b) {
      mbar_init(&red_full[b], kMmaWarps);
      mbar_init(&red_empty[b], 1);
    }
    mbar_init(x_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_tail);
    if (Fmt == kNvf4) tma_prefetch_desc(&tmap_sf);
  }
  __syncthreads();
  // The second kernel starts while the first one runs: what it reads before it
  // waits (choices, routing weights and weights) was there before the first, which
  // waited for every kernel before it ahead of letting this one start.
  if (!Down) grid_dependency_wait();
  bool ok = true;
  if (warp == 0 && !Down && elect_one_lane()) copy_tokens(p, xs, x_bar);
  if (p.slots <= 32) {
    if (warp == kTmaWarp) build_route_32<Down>(r, p, lane);
  } else {
    if (warp == kTmaWarp) count_route(r, p, lane);
    if (warp == kEpiWarp) place_route<Down>(r, p, lane);
  }
  if (!Down && warp < kMmaWarps) ok = convert_tokens<Fmt, kMmaWarps>(p, xs, r, x_bar, warp, lane);
  // the routing and the tokens are there; who loads needs only the first, which
  // that warp has
  if (warp == kTmaWarp) {
    __syncwarp();
    asm volatile("bar.arrive 3, %0;" ::"n"(S::kThreads) : "memory");
  } else {
    asm volatile("bar.sync 3, %0;" ::"n"(S::kThreads) : "memory");
  }
  const int chunks = *r.chunks;
  const int units = chunks * p.tiles;
  const int k_stages = (p.k_blocks + kSlices - 1) / kSlices;
  const int step = static_cast<int>(gridDim.x);
  UnitWalk walk{};

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    if (!elect_one_lane()) return;
    const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
    int64_t issued = 0;
    int stage = 0;
    uint32_t phase = 0;
    // the loads of K stage ks of a unit: weights, or activations
    auto load = [&](int ks, int st, int e, bool weights, bool acts) {
      uint8_t* dst = smem + st * p.stage_bytes;
      uint64_t* bar = &full_bar[st];
      const int b0 = ks * kSlices;
      const int h_bytes = Down ? r.n[walk.u] * H::kBytes : 0;
      if (weights) {
        const int row = e * p.w_rows + walk.tile * kTileRows;
        const bool whole = b0 + kSlices <= p.full_blocks;
        const int n = whole ? kSlices : min(kSlices, p.k_blocks - b0);
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * (S::kW / kSlices) + S::kS + h_bytes));
#pragma unroll
        for (int g = 0; g < (Gated ? 2 : 1); ++g) {
          uint8_t* to = dst + g * kSlices * S::kBlockW;
          if (whole) {
            tma_load_3d(&tmap_w, bar, to, 0, row + g * p.up0, b0, stream);
          } else {
            for (int j = 0; j < n; ++j)
              tma_load_2d(&tmap_tail, bar, to + j * S::kBlockW, (b0 + j) * 128, row + g * p.up0,
                          stream);
          }
          if (Fmt == kNvf4)
            tma_load_2d(&tmap_sf, bar, dst + S::kW + g * kSlices * 2048, 0,
                        (e * p.sf_rows + (walk.tile >> 2) + g * (p.up0 >> 7)) * p.k_tiles + 4 * b0,
                        keep);
        }
      }
      if (Down && acts)
        bulk_load_g2s(dst + S::kW + S::kS,
                      p.h + (static_cast<int64_t>(ks) * p.slots + r.first[walk.u]) * H::kBytes,
                      static_cast<uint32_t>(h_bytes), bar, keep);
    };
    int64_t ahead = 0;
    if (Down) {
      // the first stages' weights before the first kernel has finished
      for (int pass = 0; pass < 2; ++pass) {
        int st = 0;
        walk.start(blockIdx.x, step, chunks);
        for (; walk.tile < p.tiles && units > 0 && st < p.stages; walk.next()) {
          const int e = r.expert[walk.u];
          for (int ks = 0; ks < k_stages && st < p.stages; ++ks, ++st)
            load(ks, st, e, pass == 0, pass == 1);
        }
        ahead = st;
        if (pass == 0) grid_dependency_wait();
      }
    }
    walk.start(blockIdx.x, step, chunks);
    for (; walk.tile < p.tiles && units > 0 && ok; walk.next()) {
      const int e = r.expert[walk.u];
      for (int ks = 0; ks < k_stages; ++ks) {
        if (issued >= ahead) {
          ok = mbar_wait_abortable(&empty_bar[stage], phase ^ 1, p.timeout_ns, p.status,
                                   abort_flag);
          if (!ok) break;
          load(ks, stage, e, true, true);
        }
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // (behind this kernel's wait, never ahead of it: the next kernel reads inputs of the
    // call before its own)
    grid_launch_dependents();
    if (!ok) *abort_flag = 1;
    // the copies land before the CTA goes away, whoever gave up
    const int64_t first = issued > p.stages ? issued - p.stages : 0;
    for (int64_t i = first; i < issued; ++i)
      mbar_wait(&full_bar[i % p.stages], static_cast<uint32_t>((i / p.stages) & 1), p.timeout_ns,
                p.status);
    if (!Down && ok && chunks > 0) prefetch_next<Fmt>(p, r, chunks, step);
    if (!Down && p.K >= 8) mbar_wait(x_bar, 0, p.timeout_ns, p.status);
    return;
  }

  if (warp >= kEpiWarp) {
    // ------------------------------------------------------------ epilogue
    // The CTA's i-th unit is this warp's where i = mine modulo kEpiWarps; lane =
    // row of the tile.
    const int mine = warp - kEpiWarp;
    const float* all = red + mine * kMmaWarps * 4 * 32;
    uint32_t phase = 0;
    walk.start(blockIdx.x + mine * step, kEpiWarps * step, chunks);
    for (; walk.tile < p.tiles && units > 0; walk.next(), phase ^= 1) {
      const int tile = walk.tile, u = walk.u;
      const int e = r.expert[u], n = r.n[u], first = r.first[u];
      const int row = tile * kTileRows + lane;
      const bool there = row < p.rows;
      // the rows' scales and biases, on their way while the unit is multiplied
      float of_row[2] = {1.0f, 1.0f}, bias[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < (Gated ? 2 : 1); ++h) {
        if (Fmt == kNvf4 && there) of_row[h] = __ldg(p.row_w + e * p.stride_row + row + h * p.up0);
        if (p.bias && there) bias[h] = as_f32(p.bias, e * p.stride_bias + row + h * p.up0, p.bf16);
      }
      const bool got = mbar_wait_abortable(&red_full[mine], phase, p.timeout_ns, p.status,
                                           abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        *abort_flag = 1;
        break;
      }
      // the sum of row `lane` (of row group pair h) for the unit's slot j
      auto total = [&](int h, int j) {
        const float* at = all + ((2 * h + (lane >> 4)) * 4 + (j & 1) + 2 * ((lane >> 3) & 1)) * 32 +
                          (lane & 7) * 4 + (j >> 1);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < Teams * kSlices; ++k) s += at[k * RG * 4 * 32];
        return s;
      };
      if (!Down) {
        const int ks = tile * kTileRows / H::kK, in_stage = tile * kTileRows % H::kK;
        for (int j = 0; j < n; ++j) {
          const int pos = first + j;
          const float fx = r.fx[r.of[pos]];
          float v = scaled_sum(total(0, j), of_row[0], fx, bias[0]);
          if (Gated) {
            const float up = scaled_sum(total(1, j), of_row[1], fx, bias[1]);
            v = silu(v) * up;
          } else {
            v = gelu2(make_float2(v, v)).x;
          }
          if (!there) v = 0.0f;
          const uint32_t bits = __float_as_uint(v) & 0x7FFFFFFFu;
          const uint32_t most = __reduce_max_sync(0xffffffffu, bits < 0x7F800000u ? bits : 0u);
          float inv;
          const float f = half_factor(__uint_as_float(most), inv);
          uint8_t* to = p.h + (static_cast<int64_t>(ks) * p.slots + pos) * H::kBytes;
          // the value and what is left of it (of infinities and NaNs nothing)
          const uint32_t hi = F16::pack(v * f, 0.0f) & 0xFFFFu;
          const float rest = (hi & 0x7FFFu) < F16::kInf ? fmaf(v, f, -F16::one(hi)) : 0.0f;
          uint16_t* at = reinterpret_cast<uint16_t*>(to) + in_stage + place_of<Fmt>(lane);
          at[0] = static_cast<uint16_t>(hi);
          at[H::kRest / 2] = static_cast<uint16_t>(F16::pack(rest, 0.0f));
          if (lane == 0) reinterpret_cast<float*>(to + H::kScales)[in_stage / 32] = inv;
          if (tile == p.tiles - 1)  // zeros to the end of the last stage
            for (int i = in_stage + 32; i < H::kK; i += 32) {
              reinterpret_cast<uint16_t*>(to)[i + lane] = 0;
              reinterpret_cast<uint16_t*>(to)[H::kRest / 2 + i + lane] = 0;
              if (lane == 0) reinterpret_cast<float*>(to + H::kScales)[i / 32] = 0.0f;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&red_empty[mine]);
      } else {
        for (int j = 0; j < n; ++j) {
          const float v = fmaf(total(0, j) + total(0, j + kMaxChunkH), of_row[0], bias[0]);
          if (there) p.part[r.of[first + j] * p.part_pitch + row] = v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&red_empty[mine]);
      }
    }
    return;
  }

  // ------------------------------------------------------------------- MMAs
  const int g = lane >> 2, q = lane & 3;
  const int group = warp % RG, slice = warp % kTeamWarps / RG, team = warp / kTeamWarps;
  // ldmatrix: lanes 8 i .. 8 i + 7 give the rows of matrix i, which are (rows 0-7
  // of the group, a piece), (rows 8-15, that piece), and of the next piece
  const int mat = lane >> 3, mrow = lane & 7;
  const uint32_t smem0 = smem_addr(smem);
  // this warp's weights in a stage: its half (gate or up), block and rows
  const uint32_t a_base = smem0 +
      static_cast<uint32_t>(((group >> 1) * kSlices + slice) * S::kBlockW +
                            ((group & 1) * 16 + mrow + 8 * (mat & 1)) * 128);
  // stages go to the teams in turn: `skip` of the unit's come before this team's first
  int stage = Teams == 1 ? 0 : team, buf = 0, skip = stage;
  uint32_t phase = 0, buf_phase = 0;
  if (!ok) *abort_flag = 1;
  // FP8: the scales of the unit's weight blocks that this warp will meet, those
  // of stage ks in lane ks, for the group's first and last row (a group may
  // straddle two blocks); loaded a unit ahead.
  float sw0 = 0.0f, sw1 = 0.0f, sw0_next = 0.0f, sw1_next = 0.0f;
  const int group_row = (Gated && group >= 2 ? p.up0 - 32 : 0) + group * 16;
  const int group_end = p.rows - 1 + (Gated && group >= 2 ? p.up0 : 0);
  auto load_sw = [&](const UnitWalk& w, int ks0) {
    if (Fmt != kFp8 || w.tile >= p.tiles) return;
    const int row = group_row + w.tile * kTileRows;
    const int kb = min((ks0 + lane) * kSlices + slice, p.k_blocks - 1);
    const float* sw = p.sw + r.expert[w.u] * p.stride_sw + kb;
    sw0_next = __ldg(sw + static_cast<int64_t>(min(row, group_end) >> 7) * p.lds_w);
    sw1_next = __ldg(sw + static_cast<int64_t>(min(row + 15, group_end) >> 7) * p.lds_w);
  };
  walk.start(blockIdx.x, step, chunks);
  if (units > 0) load_sw(walk, 0);
  while (ok && walk.tile < p.tiles && units > 0) {
    const int tile = walk.tile, n = r.n[walk.u], first = r.first[walk.u];
    // this lane's column of the activations, and its two columns of the sums
    // (past the last: the last); of h, what is left in columns 4 ..
    const int col = min(Down ? g & 3 : g, n - 1);
    const uint32_t b_base =
        Down ? smem0 + static_cast<uint32_t>(S::kW + S::kS + col * H::kBytes + (g >> 2) * H::kRest +
                                             slice * S::kBlockK * 2 + q * 16)
             : smem_addr(xs) + static_cast<uint32_t>(r.of[first + col] * p.x_pitch + q * 16);
    const uint32_t h_base = smem0 + static_cast<uint32_t>(S::kW + S::kS + H::kScales +
                                                          slice * (S::kBlockK / 32) * 4);
    const uint32_t h0 = h_base + static_cast<uint32_t>(min(2 * q & 3, n - 1) * H::kBytes);
    const uint32_t h1 = h_base + static_cast<uint32_t>(min((2 * q + 1) & 3, n - 1) * H::kBytes);
    sw0 = sw0_next, sw1 = sw1_next;
    walk.next();
    load_sw(walk, 0);
    const int row_g = group_row + tile * kTileRows;
    const bool second_a = Fmt == kFp8 && (row_g + g) >> 7 != row_g >> 7;
    const bool second_b = Fmt == kFp8 && (row_g + g + 8) >> 7 != row_g >> 7;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int sw_at = 0;
    for (int ks = skip; ks < k_stages; ks += Teams) {
      if (Fmt == kFp8 && ks - sw_at >= 32) {  // beyond the 32 that lanes hold
        sw_at += 32;
        const float keep0 = sw0_next, keep1 = sw1_next;
        UnitWalk now = walk;
        now.tile = tile;
        now.u = walk.u - walk.d_u;
        if (now.u < 0) now.u += walk.chunks;
        load_sw(now, sw_at);
        sw0 = sw0_next, sw1 = sw1_next, sw0_next = keep0, sw1_next = keep1;
      }
      const int kb = ks * kSlices + slice;
      ok = __all_sync(0xffffffffu, mbar_wait_abortable(&full_bar[stage], phase, p.timeout_ns,
                                                       p.status, abort_flag));
      if (!ok) break;
      float sa = 1.0f, sb = 1.0f;
      if (Fmt == kFp8) {
        const float s0 = __shfl_sync(0xffffffffu, sw0, ks & 31);
        const float s1 = __shfl_sync(0xffffffffu, sw1, ks & 31);
        sa = second_a ? s1 : s0;
        sb = second_b ? s1 : s0;
      }
      if (kb < p.k_blocks) {
        const uint32_t at = static_cast<uint32_t>(stage * p.stage_bytes);
        const uint32_t b_at = Down ? b_base + at : b_base + static_cast<uint32_t>(kb * S::kBlockK * 2);
        uint32_t w[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
          ldmatrix4(w[m], a_base + at + (((2 * m + (mat >> 1)) ^ mrow) << 4));
        if (Fmt == kFp8) {
          uint4 b[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) b[m] = ld_shared4(b_at + m * 64);
          float c[Down ? 4 : 2][4];
#pragma unroll
          for (int m = 0; m < (Down ? 4 : 2); ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[m][i] = 0.0f;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) e4m3x4_to_f16(w[m][i], a[2 * i], a[2 * i + 1]);
            float(&d)[4] = c[Down ? m : m & 1];
            mma_f16(d, a[0], a[2], a[1], a[3], b[m].x, b[m].y);
            mma_f16(d, a[4], a[6], a[5], a[7], b[m].z, b[m].w);
          }
          if (Down) {
            const uint4 u0 = ld_shared4(h0 + at), u1 = ld_shared4(h1 + at);
            const uint32_t v0[4] = {u0.x, u0.y, u0.z, u0.w}, v1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = 0.0f;
#pragma unroll
              for (int m = 0; m < 4; ++m)
                v = fmaf(c[Down ? m : 0][i], __uint_as_float(i & 1 ? v1[m] : v0[m]), v);
              acc[i] = fmaf(v, i < 2 ? sa : sb, acc[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[i] = fmaf(c[0][i] + c[1][i], i < 2 ? sa : sb, acc[i]);
          }
        } else {
          // this lane's scale words: rows g and g + 8 of the group, four blocks each,
          // of which its codes lie in blocks q / 2 and 2 + q / 2
          const uint32_t sf = smem0 + at +
              static_cast<uint32_t>(S::kW + ((group >> 1) * kSlices + slice) * 2048 +
                                    ((group & 1) * 16 + g) * 16 + (tile & 3) * 4);
          // (a scale tile past the last is another's: its codes are zeros, NaNs not)
          if (p.k_tiles - 4 * kb < 4) {
            for (int mm = p.k_tiles - 4 * kb; mm < 4; ++mm) {
              st_shared1(sf + mm * 512, 0u);
              st_shared1(sf + mm * 512 + 128, 0u);
            }
            fence_proxy_async_smem();  // before the next copy into this stage
          }
          float c[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
          for (int mm = 0; mm < 4; ++mm) {
            uint32_t sg[2], sh[2];
            scale_pairs(ld_shared1(sf + mm * 512), q >> 1, sg);
            scale_pairs(ld_shared1(sf + mm * 512 + 128), q >> 1, sh);
            uint32_t hv0[2], hv1[2];
            if (Down) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                hv0[i] = ld_shared1(h0 + at + (2 * mm + i) * 4);
                hv1[i] = ld_shared1(h1 + at + (2 * mm + i) * 4);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 b = ld_shared4(b_at + (2 * mm + i) * 64);
              uint32_t x[4], y[4];
              e2m1x8_to_f16x2x4(w[mm][2 * i], x);
              e2m1x8_to_f16x2x4(w[mm][2 * i + 1], y);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = mul_half2(x[k], sg[i]), y[k] = mul_half2(y[k], sh[i]);
              if (Down)
#pragma unroll
                for (int k = 0; k < 4; ++k) c[i][k] = 0.0f;
              mma_f16(c[i], x[0], y[0], x[1], y[1], b.x, b.y);
              mma_f16(c[i], x[2], y[2], x[3], y[3], b.z, b.w);
            }
            if (Down) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                acc[k] = fmaf(c[1][k], __uint_as_float(k & 1 ? hv1[1] : hv0[1]),
                              fmaf(c[0][k], __uint_as_float(k & 1 ? hv1[0] : hv0[0]), acc[k]));
            }
          }
          if (!Down)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += c[0][k] + c[1][k];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[stage]);
      stage += Teams;
      if (stage >= p.stages) {
        stage -= p.stages;
        phase ^= 1;
      }
    }
    if (Teams > 1) skip = (skip + k_stages) & 1;
    // the slices' sums go to the unit's epilogue warp
    if (ok)
      ok = __all_sync(0xffffffffu, mbar_wait_abortable(&red_empty[buf], buf_phase ^ 1, p.timeout_ns,
                                                       p.status, abort_flag));
    if (!ok) {
      *abort_flag = 1;
      break;
    }
    float* mine = red + (buf * kMmaWarps + warp) * 4 * 32 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[i * 32] = acc[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&red_full[buf]);
    if (++buf == kEpiWarps) {
      buf = 0;
      buf_phase ^= 1;
    }
  }
}

// D[t,:] = the sum over j, in order, of weights[t,j] * part[t top_k + j,:] (choices
// that are dropped have no part).  A kernel of its own: added by whichever unit of the
// second product finished a token's last slot, a CTA that was late did the most of it
// and got later (16 tokens, gated NVF4: the last was at it 30 us after the others).
constexpr int kSumThreads = 128;
struct SumParams {
  const int32_t* ids;
  const float* weights;
  int top_k, count, out, bf16;
  const float* part;
  int64_t part_pitch;
  uint16_t* D;
  int64_t ldd;
};
__global__ void __launch_bounds__(kSumThreads) moe_sum_kernel(const __grid_constant__ SumParams p) {
  const int n = (static_cast<int>(blockIdx.x) * kSumThreads + static_cast<int>(threadIdx.x)) * 2;
  const int s0 = static_cast<int>(blockIdx.y) * p.top_k;
  // (choices and weights were there before the layer's first kernel)
  int e[8];
  float w[8];
  auto choices = [&](int j0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = j0 + j < p.top_k ? __ldg(p.ids + s0 + j0 + j) : -1;
      w[j] = p.weights && j0 + j < p.top_k ? __ldg(p.weights + s0 + j0 + j) : 1.0f;
    }
  };
  choices(0);
  grid_dependency_wait();
  grid_launch_dependents();
  if (n >= p.out) return;
  float2 y = make_float2(0.0f, 0.0f);
  for (int j0 = 0;;) {
    float2 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e[j] >= 0 && e[j] < p.count)
        v[j] = __ldcg(reinterpret_cast<const float2*>(
            p.part + (s0 + j0 + j) * p.part_pitch + n));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e[j] >= 0 && e[j] < p.count) {
        y.x = fmaf(w[j], v[j].x, y.x);
        y.y = fmaf(w[j], v[j].y, y.y);
      }
    if ((j0 += 8) >= p.top_k) break;
    choices(j0);
  }
  const uint32_t d = p.bf16 ? BF16::pack(y.x, y.y) : F16::pack(y.x, y.y);
  uint16_t* to = p.D + blockIdx.y * p.ldd + n;
  if (n + 1 < p.out)
    *reinterpret_cast<uint32_t*>(to) = d;
  else
    *to = static_cast<uint16_t>(d);
}

constexpr int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Where the scratch's parts lie.
struct LayerScratch {
  int64_t h, part, bytes;
};
LayerScratch scratch_of(const MoeLayerArgs& a) {
  LayerScratch s;
  const int64_t slots = a.tokens * a.top_k;
  // (either format's: the caller names none)
  const int64_t h8 = (a.hidden + HRow<kFp8>::kK - 1) / HRow<kFp8>::kK * HRow<kFp8>::kBytes;
  const int64_t h4 = (a.hidden + HRow<kNvf4>::kK - 1) / HRow<kNvf4>::kK * HRow<kNvf4>::kBytes;
  s.h = 0;
  s.part = round_up(slots * std::max(h8, h4), 16);
  s.bytes = s.part + round_up(slots * round_up(a.out, 2) * 4, 16);
  return s;
}

// Bytes of a token in shared memory: rows are 64 bytes apart in their banks.
int64_t token_bytes(const MoeLayerArgs& a) {
  return round_up(a.width, 256) * 2 + 64;
}

cudaError_t weights_map(CUtensorMap* map, const MoeWeights& w, int64_t rows, int64_t blocks,
                        int box_blocks) {
  tc::EncodeTiledFn fn = tc::encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(w.ld), 128};
  const cuuint32_t box[3] = {128, kTileRows, static_cast<cuuint32_t>(box_blocks)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w.codes), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int Fmt, bool Down, bool Gated, int Teams>
cudaError_t run_phase(const MoeLayerArgs& a, LayerParams p, int x_bytes) {
  using S = Shape<Fmt, Down, Gated, Teams>;
  static_assert(S::kBars <= 256, "barriers");
  const MoeWeights& w = Down ? a.down : a.up;
  const int64_t n_rows = Down ? a.out : a.hidden * (Gated ? 2 : 1);
  const int64_t bytes_k = Fmt == kFp8 ? p.K : (p.K + 1) / 2;
  // Slots per unit: as many as there are tokens can meet in one expert (a token
  // that names an expert twice gets a unit more), at most an MMA's columns.
  p.chunk = static_cast<int>(std::min<int64_t>(a.tokens, Down ? kMaxChunkH : kMaxChunk));
  p.inv_chunk = (65536 + p.chunk - 1) / p.chunk;
  p.k_blocks = static_cast<int>((bytes_k + 127) / 128);
  p.full_blocks = static_cast<int>(bytes_k / 128);
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
  const int stage = static_cast<int>(
      round_up(S::kW + S::kS + (Down ? p.chunk * HRow<Fmt>::kBytes : 0), 1024));
  p.stage_bytes = stage;
  const int route = route_bytes(p.slots, p.tokens, p.count);
  const int fixed = static_cast<int>(round_up(x_bytes, 16)) + S::kRed + 256 + route + 1024;
  constexpr int kMaxSmem = Teams == 1 ? 113 * 1024 : 227 * 1024;
  p.stages = std::min(kMaxStages, (kMaxSmem - fixed) / stage);
  // (FP8's second product has three stages whatever the sizes)
  if constexpr (Teams == 1 && !(Fmt == kFp8 && Down)) {
    if (p.stages < 3) return run_phase<Fmt, Down, Gated, 2>(a, p, x_bytes);
  }
  // two teams: a slot of the ring is one team's, whose waits then see its every phase
  if (Teams == 2) p.stages &= ~1;
  if (p.stages < 2) return cudaErrorInvalidValue;
  p.off_x = p.stages * stage;
  p.off_red = p.off_x + static_cast<int>(round_up(x_bytes, 16));
  p.off_route = p.off_red + S::kRed + 256;
  const int smem = p.off_route + route + 1024;

  CUtensorMap tw{}, tt{}, ts{};
  const int64_t all_rows = (a.count - 1) * pitch + n_rows;
  cudaError_t e = cudaSuccess;
  const bool whole = p.full_blocks >= S::kSlices;  // some stages' blocks
  if (whole) {
    e = weights_map(&tw, w, all_rows, p.full_blocks, S::kSlices);
    if (e != cudaSuccess) return e;
  }
  if (!whole || p.full_blocks < p.k_blocks || p.k_blocks % S::kSlices != 0) {
    e = tc::encode_map_2d(&tt, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, all_rows, bytes_k, w.ld,
                          kTileRows, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  } else {
    tt = tw;  // not used
  }
  if (!whole) tw = tt;
  ts = tw;  // not used by FP8
  if (Fmt == kNvf4) {
    e = tc::encode_map_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_UINT32, w.scales,
                          static_cast<int64_t>(p.sf_rows) * p.k_tiles * a.count, 128, 512,
                          4 * S::kSlices, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  auto kern = moe_layer_kernel<Fmt, Down, Gated, Teams>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};
  e = once_per_device(attr_set, dev, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(p.slots) * p.tiles;
  const int64_t ctas = static_cast<int64_t>(a.sm_count) * (Teams == 1 ? 2 : 1);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(most, ctas));
  e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads),
                       static_cast<size_t>(smem), a.stream, tw, tt, ts, p);
  count_launches(1);
  return e;
}

template <int Fmt>
cudaError_t run_layer(const MoeLayerArgs& a, LayerParams p, int x_bytes) {
  p.K = static_cast<int>(a.width);
  p.rows = static_cast<int>(a.hidden);
  p.up0 = static_cast<int>(a.hidden);
  p.next_w = static_cast<const uint8_t*>(a.down.codes);
  p.next_ld = a.down.ld;
  p.next_stride = a.down.stride;
  p.next_bytes = static_cast<int>(Fmt == kFp8 ? a.hidden : (a.hidden + 1) / 2);
  p.next_rows = static_cast<int>(a.out);
  p.next_k_tiles = static_cast<int>((a.hidden + 63) / 64);
  p.next_sf = static_cast<const uint8_t*>(a.down.scales);
  p.next_sf_stride = (a.out + 127) / 128 * p.next_k_tiles * 512;
  const cudaError_t e = a.gated ? run_phase<Fmt, false, true, 1>(a, p, x_bytes)
                                : run_phase<Fmt, false, false, 1>(a, p, x_bytes);
  if (e != cudaSuccess) return e;
  p.K = static_cast<int>(a.hidden);
  p.rows = static_cast<int>(a.out);
  return run_phase<Fmt, true, false, 1>(a, p, 0);
}

cudaError_t run_sum(const MoeLayerArgs& a, const LayerParams& p) {
  const SumParams q = {p.ids,  a.weights, p.top_k,      p.count,
                       static_cast<int>(a.out), a.bf16, p.part, p.part_pitch,
                       static_cast<uint16_t*>(a.D), a.ldd};
  const dim3 grid(static_cast<unsigned>((a.out + 2 * kSumThreads - 1) / (2 * kSumThreads)),
                  static_cast<unsigned>(p.tokens));
  const cudaError_t e = launch_dependent(moe_sum_kernel, grid, dim3(kSumThreads), 0, a.stream, q);
  count_launches(1);
  return e;
}

}  // namespace

int64_t moe_layer_scratch(const MoeLayerArgs& a) { return scratch_of(a).bytes; }

// What is left of a CTA's shared memory beside a ring of two stages, its sums
// and the barriers.
bool moe_layer_fits(const MoeLayerArgs& a) {
  const int64_t slots = a.tokens * a.top_k;
  return slots <= kMaxLayerSlots &&
         a.tokens * token_bytes(a) + route_bytes(slots, a.tokens, a.count) <= 150 * 1024;
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
  p.inv_top_k = ((1 << 20) + p.top_k - 1) / p.top_k;
  p.bf16 = a.bf16;
  p.X = static_cast<const uint16_t*>(a.X);
  p.ldx = a.ldx;
  p.x_pitch = static_cast<int>(token_bytes(a));
  p.h = base + s.h;
  p.part = reinterpret_cast<float*>(base + s.part);
  p.part_pitch = round_up(a.out, 2);
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  const int x_bytes = static_cast<int>(a.tokens * token_bytes(a));
  const cudaError_t e = a.nvf4 ? run_layer<kNvf4>(a, p, x_bytes) : run_layer<kFp8>(a, p, x_bytes);
  return e == cudaSuccess ? run_sum(a, p) : e;
}

}  // namespace dg
