// Experts' row segments on the device: how many tiles each has, for the
// products that walk them.
#pragma once

#include <stdint.h>

#include "dg.h"

namespace dg {

constexpr int kMaxTiles = 1 << 30;  // tile numbers are 32-bit, and a walk steps past the last

// pre[e] = row blocks of `rows` rows in the segments before e (off[e] .. off[e + 1] - 1,
// clamped offsets in shared memory), for e = 0 .. count; by one warp.
//
// Segments in order have at most one part-filled block each, and the host has checked that
// those make no more than kMaxTiles tiles.  Offsets that go back and forth make segments
// that overlap, up to count / 2 times all rows (512 experts, 8192 rows in blocks of 8 and
// 4096 tiles of columns: 2^31 tiles): the count stops at `most` row blocks, kMaxTiles by the
// tiles of columns, what lies behind it is not computed, and `report` records it in the
// status word.
__device__ __forceinline__ void count_row_blocks(const int* off, int* pre, int count, int rows,
                                                 uint32_t most, bool report, int* status,
                                                 int lane) {
  uint32_t run = 0;
  bool over = false;
  if (lane == 0) pre[0] = 0;
  for (int e0 = 0; e0 < count; e0 += 32) {
    const int e = e0 + lane;
    // (32 of them and `most` stay below 2^32)
    uint32_t v = 0;
    if (e < count) v = min((max(off[e + 1] - off[e], 0) + rows - 1) / rows, 1 << 26);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    over |= run + v > most;
    v = min(run + v, most);
    if (e < count) pre[e + 1] = static_cast<int>(v);
    run = __shfl_sync(0xffffffffu, v, 31);
  }
  if (report && __any_sync(0xffffffffu, over) && lane == 0)
    atomicExch(status, static_cast<int>(DG_ERR_INVALID_ARG));
}

}  // namespace dg
