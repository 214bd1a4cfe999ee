// chunk.cuh -- which work a CTA of the attention of chunks over a paged cache takes,
// and which keys its rows see.
//
// An item is a tile of a sequence's new tokens and a head; its cost is its key
// tiles and ChunkCost::start for its beginning and end.  The items of all sequences form
// a list, heads innermost, and CTA c takes the c-th of `count` equal parts of the
// list's cost: it continues an item that others began, takes whole ones, and begins
// one that others end.  So CTAs are equally loaded whatever the lengths, which only
// the device knows, and an item is cut only where a CTA's part ends (and not within
// ChunkCost::snap tiles of its ends).  Each CTA finds its part by itself, from the costs of
// all items, which its threads sum: it knows it 3.7 us after its start (a kernel of one
// block in front that did it for all, its successor's set-up beside it, took 5.5 by itself).  Parts of
// cut items leave normalised outputs and log-sum-exps in the workspace, two slots
// per CTA, for the join.
#pragma once

#include "debug_checks.cuh"
#include "paged.cuh"

namespace jvp {

struct ChunkSequence {
  int r0, len, keys;  // first row, new tokens, positions
  int items;          // tiles of tokens
};
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
  s.items = static_cast<int>((static_cast<unsigned>(s.len) + rows - 1u) / rows);
  return s;
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
  __device__ __forceinline__ ChunkKeys() {}
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
// Tokens of an item: up to query_tiles tiles of rows of tok tokens.
__device__ __forceinline__ int chunk_step(const ChunkParams& p) { return p.query_tiles * p.tok; }
// Key tiles by which an item is cut: those of its first tile of rows (a second one
// may have one more, which goes with the last part).
template <int TILE>
__device__ __forceinline__ int chunk_tiles(const ChunkParams& p, const ChunkSequence& s, int item,
                                           ChunkKeys<TILE>* keys) {
  const int past = s.keys - s.len, tok0 = item * chunk_step(p);
  const int toks = min(s.len - tok0, chunk_step(p));
  *keys = ChunkKeys<TILE>(p, past + tok0, past + tok0 + toks - 1);
  return keys->tiles(past + tok0 + min(toks, p.tok) - 1);
}

// Shared memory of the division (the tiles' space, before they are copied).
constexpr int kChunkSeqs = 2048;  // sequences at a time
struct ChunkScratch {
  long long part[32];
  int4 plan[2];         // where the CTA's part begins and ends
  long long cut_first;  // of the item in which it ends: its first position of the list
  int cut_cost;
  int first[kChunkSeqs + 1], r0[kChunkSeqs], len[kChunkSeqs], keys[kChunkSeqs];
};
// Exclusive sum over the block, and the total.
template <int THREADS>
__device__ __forceinline__ long long chunk_block_sum(long long x, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before + incl - x;
}

// Where part k of `count` of a list of cost W begins.
__device__ __forceinline__ long long chunk_position(long long W, int count, int k) {
  // 32-bit arithmetic where it does: a 64-bit division takes a fifth of a microsecond
  if (W < (1ll << 31)) {
    const unsigned w = static_cast<unsigned>(W), n = static_cast<unsigned>(count);
    return w / n * k + w % n * k / n;
  }
  return W / count * k + W % count * k / count;
}

// A CTA's part: where it begins and ends (sequence, item, head, key tile), and of the item
// in which it ends.
struct ChunkSpan {
  int4 start, end;
  long long W, cut_first;  // the list's cost; where the item begins
  int count, cut_cost;     // parts; the item's cost
};
// The part of CTA blockIdx.x; false if it has none.  Executed by the whole block.  CTA 0
// reports bad offsets and lengths.
template <int TILE, int THREADS>
__device__ __forceinline__ bool chunk_divide(const ChunkParams& p, ChunkScratch* sh,
                                             ChunkSpan* span) {
  const int tid = static_cast<int>(threadIdx.x), B = p.c.B, step = chunk_step(p);
  constexpr ChunkCost kCost = chunk_cost(TILE);
  bool bad = false, over = false;
  int b0 = 0, nb = 0;  // sequences in shared memory
  // A thread takes neighbouring sequences, and neighbouring items, so that there is one
  // sum over the block for each, however many there are.
  auto load_round = [&](int from) {  // returns their items
    b0 = from, nb = min(B - from, kChunkSeqs);
    const int per = (nb + THREADS - 1) / THREADS, i0 = min(nb, tid * per), i1 = min(nb, i0 + per);
    int items = 0;
    for (int i = i0; i < i1; ++i) {
      const ChunkSequence s = chunk_sequence(p, step, b0 + i, &bad);
      sh->first[i] = items, sh->r0[i] = s.r0, sh->len[i] = s.len, sh->keys[i] = s.keys;
      items += s.items;
    }
    long long total;
    long long before = chunk_block_sum<THREADS>(items, sh->part, &total);
    // More items than rows and sequences: sequences overlap, however good the offsets of
    // each, and none is taken (the sum may pass an int, and the work any bound).
    over |= total > static_cast<long long>(p.T) + nb;
    if (over) bad = true, before = total = 0;
    for (int i = i0; i < i1; ++i) sh->first[i] = over ? 0 : sh->first[i] + static_cast<int>(before);
    if (tid == 0) sh->first[nb] = static_cast<int>(total);
    __syncthreads();
    return static_cast<int>(total);
  };
  int b = 0, in_seq = 0;  // of an item
  auto seek = [&](int i) {  // item i of the round: the last sequence with first <= i
    int lo = 0, hi = nb;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh->first[mid] <= i) lo = mid;
      else hi = mid;
    }
    b = lo;
  };
  auto cost_of = [&](int i) {  // of item i, the one sought or behind it
    while (sh->first[b + 1] <= i) ++b;
    in_seq = i - sh->first[b];
    ChunkSequence s;
    s.r0 = sh->r0[b], s.len = sh->len[b], s.keys = sh->keys[b];
    ChunkKeys<TILE> keys;
    return kCost.start + chunk_tiles(p, s, in_seq, &keys);
  };
  const int c = static_cast<int>(blockIdx.x);
  int i0 = 0, i1 = 0, count = 0;  // the thread's items; parts
  // the thread's items' cost, that of the items in front, of all, and with all heads
  long long mine = 0, before = 0, all = 0, W = 0;
  // All costs first, then the items in which the part begins and ends.  (One loop for
  // both, and short ones: a kernel's first pass over its instructions is slow.)
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      W = over ? 0 : all * p.heads;
      const long long parts = W / kCost.least;
      count = static_cast<int>(W == 0 ? 0 : parts < 1 ? 1 : parts > p.grid ? p.grid : parts);
      if (c == 0 && bad) atomicOr(p.c.status, kStatusIndex);
      if (c >= count) {
        if (tid == 0) p.ws_item[c] = make_int4(0, 0, 0, 0);
        return false;
      }
      if (tid == 0 && c + 1 == count) sh->plan[1] = make_int4(B, 0, 0, 0);
      if (B > kChunkSeqs) all = 0;
    }
#pragma unroll 1
    for (int from = 0; from < B; from += kChunkSeqs) {
      if (pass == 0 || B > kChunkSeqs) {
        const int I = load_round(from);
        const int per = static_cast<int>((static_cast<unsigned>(I) + THREADS - 1) / THREADS);
        i0 = static_cast<int>(min(static_cast<long long>(I), static_cast<long long>(tid) * per));
        i1 = min(I, i0 + per);
        mine = 0;
        if (i0 < i1) seek(i0);
#pragma unroll 1
        for (int i = i0; i < i1; ++i) mine += cost_of(i);
        long long total;
        before = all + chunk_block_sum<THREADS>(mine, sh->part, &total);
        all += total;
      }
      if (pass == 0) continue;
#pragma unroll 1
      for (int which = 0; which < (c + 1 < count ? 2 : 1); ++which) {
        const long long x = chunk_position(W, count, c + which);
        long long first = before * p.heads;
        if (x < first || x >= first + mine * p.heads) continue;
        // the item at x is the thread's
        if (i1 - i0 > 1) seek(i0);
        int i = i0, cost;
#pragma unroll 1
        while (cost = cost_of(i), x >= first + static_cast<long long>(cost) * p.heads)
          first += static_cast<long long>(cost) * p.heads, ++i;
        const long long in = x - first;
        const int h = W < (1ll << 31)
                          ? static_cast<int>(static_cast<unsigned>(in) / static_cast<unsigned>(cost))
                          : static_cast<int>(in / cost);
        const int d = static_cast<int>(in - static_cast<long long>(h) * cost);
        int4 y = make_int4(b0 + b, in_seq, h, 0);
        if (p.cut ? d < kCost.start + kCost.snap : d == 0) {
        } else if (p.cut && cost - d >= kCost.snap) {
          y.w = d - kCost.start;
          if (which) sh->cut_first = x - d, sh->cut_cost = cost;
        } else if (++y.z == p.heads) {  // the next item is the first of the next part
          y.y += 1, y.z = 0;
          bool ignore = false;
          while (y.x < B && y.y >= chunk_sequence(p, step, y.x, &ignore).items) y.x += 1, y.y = 0;
        }
        sh->plan[which] = y;
      }
      __syncthreads();
    }
  }
  span->start = sh->plan[0], span->end = sh->plan[1];
  span->W = W, span->count = count;
  span->cut_first = sh->cut_first, span->cut_cost = sh->cut_cost;
  __syncthreads();  // the scratch has been read
  return true;
}
// Names for the join the item that the CTA begins and others end.  One thread.
template <int TILE>
__device__ __forceinline__ void chunk_name(const ChunkParams& p, const ChunkSpan& x) {
  const int c = static_cast<int>(blockIdx.x);
  const int4 &start = x.start, &end = x.end;
  int4 item = make_int4(0, 0, 0, 0);
  const bool goes_on = start.x == end.x && start.y == end.y && start.z == end.z && start.w > 0;
  if (end.w > 0 && !goes_on) {
    // the CTA in whose part its last unit lies, unless that part begins so near the
    // item's end that it leaves it to the one before
    const long long last = x.cut_first + x.cut_cost - 1;
    // (near it, within the rounding of fp32)
    int c1 = min(static_cast<int>(static_cast<float>(last) / static_cast<float>(x.W) * x.count),
                 x.count - 1);
    while (chunk_position(x.W, x.count, c1) > last) --c1;
    while (c1 + 1 < x.count && chunk_position(x.W, x.count, c1 + 1) <= last) ++c1;
    if (last + 1 - chunk_position(x.W, x.count, c1) < chunk_cost(TILE).snap) --c1;
    bool ignore = false;
    const int step = chunk_step(p), tok0 = end.y * step;
    const ChunkSequence s = chunk_sequence(p, step, end.x, &ignore);
    item = make_int4(c1 - c + 1, s.r0 + tok0, min(s.len - tok0, step), end.z);
  }
  p.ws_item[c] = item;
}

// A CTA's part of one item: key tiles [t0, t1) of `all`, in slot `slot` of the
// workspace (-1: it is the whole item).
template <int TILE>
struct ChunkPart {
  int b, r0, len, past, keys;  // as in the sequence; past: positions before its new tokens
  int tok0, toks, head;
  int t0, t1, all, slot;
  ChunkKeys<TILE> see;
};

// The parts of CTA blockIdx.x, one after the other.  Every warp walks for itself.
template <int TILE>
struct ChunkWalk {
  int b, item, head, t;
  int4 end;
  ChunkSequence s;
  bool more;
  __device__ __forceinline__ ChunkWalk(const ChunkParams& p, const int4& a, const int4& e) {
    end = e;
    b = a.x, item = a.y, head = a.z, t = a.w;
    more = b < p.c.B;
    bool bad = false;
    if (more) s = chunk_sequence(p, chunk_step(p), b, &bad);
  }
  __device__ __forceinline__ bool next(const ChunkParams& p, ChunkPart<TILE>* part) {
    while (more) {
      const bool last = b == end.x && item == end.y && head == end.z;
      part->all = chunk_tiles(p, s, item, &part->see);
      part->b = b, part->r0 = s.r0, part->len = s.len, part->keys = s.keys;
      part->past = s.keys - s.len;
      part->tok0 = item * chunk_step(p), part->toks = min(s.len - part->tok0, chunk_step(p));
      part->head = head;
      part->t0 = t, part->t1 = last ? end.w : part->all;
      part->slot = t > 0 ? 2 * static_cast<int>(blockIdx.x)
                         : (part->t1 < part->all ? 2 * static_cast<int>(blockIdx.x) + 1 : -1);
      if (last) {
        more = false;
      } else {
        t = 0;
        if (++head == p.heads) {
          head = 0;
          if (++item == s.items) {
            item = 0;
            bool bad = false;
            do {
              ++b;
              if (b < p.c.B) s = chunk_sequence(p, chunk_step(p), b, &bad);
            } while (b < p.c.B && s.items == 0);
            more = b < p.c.B;
          }
        }
      }
      if (part->t0 < part->t1) return true;
    }
    return false;
  }
};

}  // namespace jvp
