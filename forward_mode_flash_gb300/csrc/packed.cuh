// packed.cuh -- which rows of a packed batch a block of an attention kernel
// takes: sequence lengths live on the device, so each block finds its own.
#pragma once

#include "serve_internal.h"

namespace jvp {

struct PackedTile {
  int r0, len;  // the sequence's first row and length
  int tile;     // query tile within the sequence
};

// Query tile `u` of the list of all sequences' tiles (ceil(len / rows) each),
// for each sequence last tile first where `last_first`.  Executed by a whole
// warp; false where the list has fewer tiles.  Offsets outside 0 <= cu[b] <=
// cu[b + 1] <= T make an empty sequence and are recorded by the block u = 0.
__device__ __forceinline__ bool find_packed_tile(const int* cu, int B, int T, int rows, int u,
                                                 bool last_first, unsigned int* status,
                                                 PackedTile* out) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  bool bad = false, found = false;
  int next0 = lane < B ? __ldg(cu + lane) : 0, next1 = lane < B ? __ldg(cu + lane + 1) : 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int r0 = next0, r1 = next1;
    // (the next 32 offsets are fetched while these are summed)
    const int nb = b0 + 32 + lane;
    next0 = nb < B ? __ldg(cu + nb) : 0, next1 = nb < B ? __ldg(cu + nb + 1) : 0;
    if (r0 < 0 || r1 < r0 || r1 > T) {
      bad = true;
      r0 = r1 = 0;
    }
    const int nt = (r1 - r0 + rows - 1) / rows;
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (!found) {
      const unsigned past = __ballot_sync(0xffffffffu, base + incl > u);
      if (past) {
        found = true;
        const int src = __ffs(past) - 1;
        const int before = base + __shfl_sync(0xffffffffu, incl - nt, src);
        const int n = __shfl_sync(0xffffffffu, nt, src);
        out->r0 = __shfl_sync(0xffffffffu, r0, src);
        out->len = __shfl_sync(0xffffffffu, r1, src) - out->r0;
        out->tile = last_first ? n - 1 - (u - before) : u - before;
        if (u != 0) return true;  // block 0 goes on to check every offset
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (u == 0 && bad) atomicOr(status, kStatusIndex);
  return found;
}

}  // namespace jvp
