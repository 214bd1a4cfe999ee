// chunk.cuh -- which work a block of the attention of chunks over a paged cache
// takes, and which keys its rows see.  Lengths live on the device, so each block
// finds its own.
//
// An item is a tile of a sequence's new tokens (ROWS tokens) and a head; its keys
// are cut into pieces where that keeps the GPU busy.  With n_b key tiles of a
// sequence's items (a bound) and t_b items per head, W = heads sum t_b n_b and
// L = max(least, ceil(W / target)), each of its items is cut into S_b =
// ceil(n_b / L) pieces: equal parts, so pieces are of about L tiles however the
// lengths are spread, and nothing is cut where there are items enough.  Pieces of
// cut items number at most 2 target: S_b <= 2 n_b / L where S_b > 1.
#pragma once

#include "debug_checks.cuh"
#include "paged.cuh"

namespace jvp {

struct ChunkItem {
  int b, r0, len, past;  // sequence, its first row, new tokens, positions before them
  int keys;              // positions of the sequence
  int tok0;              // the item's first token
  int piece, pieces;     // pieces as the sequence's items are cut (S_b)
  long long slot;        // of the item's first piece for head 0, or -1: not cut
};

struct ChunkSequence {
  int r0, len, keys;
  long long items;  // tiles of tokens
  int tiles;        // key tiles of an item, at most
};

template <int TILE>
__device__ __forceinline__ ChunkSequence chunk_sequence(const ChunkParams& p, int rows, int b,
                                                        bool* bad) {
  ChunkSequence s;
  const int r0 = __ldg(p.cu + b), r1 = __ldg(p.cu + b + 1);
  s.keys = clamp_len(p.c, __ldg(p.lens + b), bad);
  s.r0 = r0, s.len = r1 - r0;
  if (r0 < 0 || r1 < r0 || r1 > p.T) {
    *bad = true;
    s.r0 = s.len = 0;
  }
  s.items = (s.len + static_cast<long long>(rows) - 1) / rows;
  long long n = (s.keys + static_cast<long long>(TILE) - 1) / TILE;
  if (p.window > 0) {  // the window's keys of `rows` tokens begin anywhere in a tile
    const long long span = static_cast<long long>(p.window) + rows - 2;
    const long long most = (span + TILE - 1) / TILE + 1 + (p.sinks + TILE - 1ll) / TILE;
    n = n < most ? n : most;
  }
  s.tiles = n < 1 ? 1 : static_cast<int>(n);
  return s;
}
// Largest number of tiles of a piece, of W tiles in all.
__device__ __forceinline__ long long chunk_piece_tiles(const ChunkParams& p, long long W) {
  if (p.least == 0) return 1ll << 40;
  const long long even = (W + p.target - 1) / p.target;
  return even > p.least ? even : p.least;
}

template <typename T>
__device__ __forceinline__ T warp_inclusive(T x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

struct ChunkScan {
  long long part[32], part2[32];
  ChunkItem item;
  int found;
};

// Unit u of the list of all sequences' (tile of tokens, piece) pairs, a
// sequence's last tokens (the longest key ranges) first.  Executed by the whole
// block; false where the list is shorter.  `first`: of the blocks with u = 0 the
// one that reports bad offsets and lengths and records the slots in use.
template <int TILE, int THREADS>
__device__ __forceinline__ bool find_chunk_item(const ChunkParams& p, int rows, int u, bool first,
                                                ChunkScan* sh, ChunkItem* out) {
  const int lane = threadIdx.x & 31;
  const int B = p.c.B;
  bool bad = false;
  // (each thread a run of sequences; up to 32 sequences: each warp for itself)
  const bool small = B <= 32;
  const int threads = small ? 32 : THREADS, me = small ? lane : static_cast<int>(threadIdx.x);
  const int per = (B + threads - 1) / threads;
  const int b_lo = min(B, me * per), b_hi = min(B, b_lo + per);
  auto block_inclusive = [&](long long x, long long* part, long long* total) {
    long long incl = warp_inclusive(x);
    if (small) {
      *total = __shfl_sync(0xffffffffu, incl, 31);
      return incl;
    }
    if (lane == 31) part[threadIdx.x >> 5] = incl;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x >> 5)) before += part[w];
      all += part[w];
    }
    __syncthreads();
    *total = all;
    return before + incl;
  };
  long long w = 0;
  ChunkSequence s{};
  for (int b = b_lo; b < b_hi; ++b) {
    s = chunk_sequence<TILE>(p, rows, b, &bad);
    w += s.items * s.tiles;
  }
  long long W;
  block_inclusive(w, sh->part, &W);
  const long long L = chunk_piece_tiles(p, W * p.heads);
  long long units = 0, cut = 0;  // of this thread's sequences: pieces, those of cut items
  for (int b = b_lo; b < b_hi; ++b) {
    if (per > 1) s = chunk_sequence<TILE>(p, rows, b, &bad);
    const long long S = (s.tiles + L - 1) / L, n = s.items * S;
    units += n;
    if (S > 1) cut += n;
  }
  long long all_units, all_cut;
  long long before = block_inclusive(units, sh->part, &all_units) - units;
  long long cut_before = block_inclusive(cut, sh->part2, &all_cut) - cut;
  if (first && u == 0) {
    if (bad) atomicOr(p.c.status, kStatusIndex);
    if (threadIdx.x == 0 && p.least > 0) *p.ws_count = static_cast<int>(all_cut * p.heads);
  }
  if (u >= all_units) return false;
  ChunkItem item{};
  const bool mine = u >= before && u < before + units;
  if (mine) {
    int b = b_lo;
    long long n = 0, S = 1;
    for (; b < b_hi; ++b) {
      if (per > 1) s = chunk_sequence<TILE>(p, rows, b, &bad);
      S = (s.tiles + L - 1) / L, n = s.items * S;
      if (u < before + n) break;
      before += n;
      if (S > 1) cut_before += n;
    }
    const long long at = u - before, back = at / S;
    item.b = b, item.r0 = s.r0, item.len = s.len, item.keys = s.keys;
    item.past = s.keys - s.len;
    item.tok0 = static_cast<int>((s.items - 1 - back) * rows);
    item.piece = static_cast<int>(at - back * S), item.pieces = static_cast<int>(S);
    item.slot = S > 1 ? (cut_before + back * S) * p.heads : -1;
  }
  if (small) {
    const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    out->b = __shfl_sync(0xffffffffu, item.b, src);
    out->r0 = __shfl_sync(0xffffffffu, item.r0, src);
    out->len = __shfl_sync(0xffffffffu, item.len, src);
    out->past = __shfl_sync(0xffffffffu, item.past, src);
    out->keys = __shfl_sync(0xffffffffu, item.keys, src);
    out->tok0 = __shfl_sync(0xffffffffu, item.tok0, src);
    out->piece = __shfl_sync(0xffffffffu, item.piece, src);
    out->pieces = __shfl_sync(0xffffffffu, item.pieces, src);
    out->slot = __shfl_sync(0xffffffffu, item.slot, src);
  } else {
    if (mine) sh->item = item;
    __syncthreads();
    *out = sh->item;
  }
  return true;
}

// The keys that the rows of an item see.  A row at position x sees [lo(x), x] and,
// before lo(x), the sinks.  Tiles are numbered in a row, those that no row of the
// item sees left out: `front` of the sinks', then, `skip` tiles on, the window's.
template <int TILE>
struct ChunkKeys {
  int window, sinks;
  int lo_first, lo_last;  // lo of the item's first and last row
  int end;                // keys of its last row
  int front, skip;
  __device__ __forceinline__ int lo(int x) const { return window > 0 ? max(0, x - window + 1) : 0; }
  // rows at positions first .. last (either may be negative: no keys)
  __device__ __forceinline__ ChunkKeys(const ChunkParams& p, int first, int last) {
    window = p.window, sinks = p.sinks;
    lo_first = lo(first), lo_last = lo(last);
    end = max(0, last + 1);
    front = (min(sinks, lo_first) + TILE - 1) / TILE;
    skip = max(0, lo_first / TILE - front);
  }
  __device__ __forceinline__ int tile(int i) const { return i >= front ? i + skip : i; }
  // tiles (numbered in a row) up to the keys of a row at position x: one at least
  __device__ __forceinline__ int tiles(int x) const { return max(1, x / TILE + 1 - skip); }
  // keys [j, j + n) are seen by no row
  __device__ __forceinline__ bool unseen(int j, int n) const {
    return j >= end || (j >= sinks && j + n <= lo_first);
  }
  __device__ __forceinline__ bool sees(int x, int j) const {
    return j <= x && (j >= lo(x) || j < sinks);
  }
};

}  // namespace jvp
