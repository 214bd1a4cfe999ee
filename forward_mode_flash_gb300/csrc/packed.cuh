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
// for each sequence last tile first where `last_first`.  Otherwise a tile's work
// goes with its sequence's length, and up to 32 sequences are taken longest
// first (16 of 90 to 1024 tokens, 8 heads, D = 64: 37.1 against 39.6 us).  The
// same over the tiles of causal sequences, last tiles of all first, is slower
// (66.0 against 63.7 us, 4 of 2048 tokens, 16/4 heads, D = 128).  Beyond 32
// sequences, and for causal ones, the offsets before the tile's sequence are
// walked, 32 at a time: every block's start takes longer with many sequences.
// Executed by a whole warp; false where the list has fewer tiles.  Offsets outside 0 <= cu[b] <=
// cu[b + 1] <= T make an empty sequence and are recorded by the block u = 0.
__device__ __forceinline__ bool find_packed_tile(const int* cu, int B, int T, int rows, int u,
                                                 bool last_first, unsigned int* status,
                                                 PackedTile* out) {
  const int lane = threadIdx.x & 31;
  if (B <= 32 && !last_first) {  // longest sequences first
    int r0 = lane < B ? __ldg(cu + lane) : 0, r1 = lane < B ? __ldg(cu + lane + 1) : 0;
    const bool wrong = r0 < 0 || r1 < r0 || r1 > T;
    if (wrong) r0 = r1 = 0;
    if (u == 0 && __any_sync(0xffffffffu, wrong) && lane == 0) atomicOr(status, kStatusIndex);
    const int nt = (r1 - r0 + rows - 1) / rows;
    // x: the smallest number with at most u tiles in sequences of more than x
    // tiles (`before` of them)
    int lo = 0, x = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(nt)));
    int before = 0;
    while (x - lo > 1) {
      const int mid = (lo + x) >> 1;
      const int n = static_cast<int>(
          __reduce_add_sync(0xffffffffu, static_cast<unsigned>(nt > mid ? nt : 0)));
      if (n > u) lo = mid;
      else x = mid, before = n;
    }
    const unsigned of_x = __ballot_sync(0xffffffffu, nt == x);
    const int k = u - before;
    if (x == 0 || k >= __popc(of_x) * x) return false;
    const int which = k / x;
    const unsigned pick = __ballot_sync(
        0xffffffffu, nt == x && __popc(of_x & ((1u << lane) - 1u)) == which);
    const int src = __ffs(pick) - 1;
    out->r0 = __shfl_sync(0xffffffffu, r0, src);
    out->len = __shfl_sync(0xffffffffu, r1, src) - out->r0;
    out->tile = k - which * x;
    return true;
  }
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
