// chunk_tc.cuh -- attention of chunks of new tokens over a paged cache on the
// tensor cores (tcgen05 + TMEM), fp16 / bf16, fp32 accumulation.
//
// The softmax, its rounding and the flow between copies, products and softmax are
// those of the kernel over packed prompts (packed_tc.cuh): 128-row query tiles of
// `tok` tokens times the query heads of a key/value head, two tiles (NQ) per CTA
// against the same ring of 128-key K/V tiles.  What differs:
//   - Key tiles are collected from pages.  SRC = kChunkBoxes: the largest power of
//     two of rows that divides a page (8 at least) is one TMA box; the lanes of the
//     copying warp each look up one box's page and issue its copy, K's and V's from
//     one lookup, made a tile ahead.  A box that no row sees, or whose page does not
//     exist, is copied from behind the last page, where TMA writes zeros.
//     SRC = kChunkRows (pages of any size) and kChunkE4M3: four more warps gather
//     the rows in 8-element pieces by asynchronous copies three half tiles ahead, one
//     thread looking up each key's place a tile ahead.  e4m3 pieces land in a staging
//     area, and the thread that copied a piece converts it (a code is exact in fp16
//     and bf16; times its scale, rounded to T as cache_read does).
//   - A row sees an interval of keys and the sinks (ChunkKeys); tiles that no row
//     sees are left out.
//   - Few tokens over long contexts have few items: their key tiles are cut into
//     pieces (chunk.cuh), whose normalised outputs and log-sum-exps a second
//     kernel joins in a fixed order.
// Keys of pages that do not exist are masked by a bit each.
#pragma once

#include "chunk.cuh"
#include "packed_tc.cuh"

namespace jvp {

// The gathering sources: threads, registers (65536 / 512 a thread: 56 + 104 + 2 * 176 =
// 4 * 128), and their shared memory behind the control block.
constexpr int chunk_threads(int NQ, ChunkSource src) {
  return packed_threads(NQ) + (src == kChunkBoxes ? 0 : 128);
}
struct ChunkPlaces {
  long long k[kChunkTile], v[kChunkTile];  // elements from the start of the cache, -1: none
  uint8_t k_scale[2][kChunkTile], v_scale[2][kChunkTile];  // by tile modulo 2
};
constexpr int kChunkAhead = 3;  // half tiles in flight
template <int D, int NQ, ChunkSource SRC>
struct ChunkLayout : PackedLayout<D, NQ> {
  using P = PackedLayout<D, NQ>;
  static constexpr int HALF_CODES = 64 * D;  // bytes of half a tile of codes
  static constexpr int OFF_PLACES = P::OFF_CTRL + 1024;
  static constexpr int OFF_STAGE = OFF_PLACES + static_cast<int>(sizeof(ChunkPlaces));
  static constexpr int BYTES = SRC == kChunkBoxes ? P::SMEM_BYTES
                               : SRC == kChunkRows
                                   ? P::SMEM_BYTES + static_cast<int>(sizeof(ChunkPlaces))
                                   : P::SMEM_BYTES + static_cast<int>(sizeof(ChunkPlaces)) +
                                         kChunkAhead * HALF_CODES;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

template <int D, int NQ, int NS>
struct ChunkCtrl {
  uint64_t q_full[2];
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t v_issued[NS], v_checked[NS];
  uint64_t s_full[2][3], p_full[2][3], o_done[2][3];
  uint64_t o_full[2];
  uint64_t staged[2];
  uint64_t drain[2];
  // By key tile modulo 16 (the copies are at most 2 NS tiles ahead of the
  // softmax), a bit for every key: its page does not exist.
  alignas(16) uint32_t missing[16][4];
  uint32_t tmem_base;
  int abort;
  int special;
};

// Asynchronous copy of BYTES, or zeros.
template <int BYTES>
__device__ __forceinline__ void chunk_copy(uint32_t dst, const void* src, bool on) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0)
                 : "memory");
}
// Two codes (as fp16 values, which hold them exactly), times the scale, rounded to T.
template <typename T>
__device__ __forceinline__ uint32_t chunk_decode(uint32_t half2, float scale) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&half2));
  return PackedElem<T>::pack(f.x * scale, f.y * scale);
}

template <typename T, int D, int NQ, ChunkSource SRC>
__global__ void __launch_bounds__(chunk_threads(NQ, SRC), SRC == kChunkBoxes ? 3 - NQ : 1)
    chunk_tc_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkParams p) {
  using L = ChunkLayout<D, NQ, SRC>;
  constexpr int BM = L::BM, BN = L::BN, NS = L::NS, NB = L::NB, KCH = L::KCH;
  constexpr int THREADS = chunk_threads(NQ, SRC);
  constexpr bool kGather = SRC != kChunkBoxes;
  constexpr int kSoftmax = kGather ? 8 : 4;  // first softmax warp
  constexpr bool kBF16 = PackedElem<T>::kBF16;
  constexpr uint32_t IDESC_S = idesc_f16(kBF16, BM, BN, false);
  constexpr uint32_t IDESC_O = idesc_f16(kBF16, BM, D, true);
  static_assert(BN == kChunkTile, "key tiles");

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using Ctrl = ChunkCtrl<D, NQ, NS>;
  static_assert(sizeof(Ctrl) <= 1024, "control block budget");
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + L::OFF_CTRL);
  // (in the query tiles' space, before they are copied)
  ChunkScan* scan = reinterpret_cast<ChunkScan*>(smem + L::OFF_V);
  volatile int* abort = &ctrl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedCache& c = p.c;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.o);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctrl->q_full[x], 1);
      for (int i = 0; i < 3; ++i) {
        mbar_init(&ctrl->s_full[x][i], 1);
        mbar_init(&ctrl->p_full[x][i], 4);  // one arrival per softmax warp of the tile
        mbar_init(&ctrl->o_done[x][i], 1);
      }
      mbar_init(&ctrl->o_full[x], 1);
      mbar_init(&ctrl->drain[x], 1);
      mbar_init(&ctrl->staged[x], 4);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&ctrl->k_full[s], kGather ? 4 : 1);  // one arrival per gathering warp
      mbar_init(&ctrl->k_empty[s], NB == 3 ? 2 : 1);  // one arrival per issuing warp
      mbar_init(&ctrl->v_full[s], kGather ? 4 : 1);
      mbar_init(&ctrl->v_empty[s], NB == 3 ? 2 : 1);
      mbar_init(&ctrl->v_issued[s], 1);
      mbar_init(&ctrl->v_checked[s], 1);
    }
    ctrl->abort = 0;
    ctrl->special = 0;
    fence_barrier_init();
  }
  __syncwarp();
  // A tile's key/value heads one behind the other: they have the same length.
  const int hk = static_cast<int>(blockIdx.x) % p.heads;
  const int u = static_cast<int>(blockIdx.x) / p.heads;
  ChunkItem it;
  if (!find_chunk_item<BN, THREADS>(p, NQ * p.tok, u, hk == 0, scan, &it)) return;
  const int tok0 = it.tok0, len = it.len, r0 = it.r0;  // first token of tile A; B follows
  const int toks = min(len - tok0, NQ * p.tok);        // tokens of the item
  const ChunkKeys<BN> keys(p, it.past + tok0, it.past + tok0 + toks - 1);
  // key tiles of the query tiles, and this piece's: A's are cut evenly, and where B
  // has more they go with the last piece
  const int all_a = keys.tiles(it.past + tok0 + min(toks, p.tok) - 1);
  const int all_b = toks > p.tok ? keys.tiles(it.past + tok0 + toks - 1) : 0;
  const int pieces = min(it.pieces, all_a);
  const int slot = it.slot < 0 ? -1 : static_cast<int>(it.slot) + it.piece * p.heads + hk;
  if (slot >= 0 && threadIdx.x == 0 && JVP_CHECK(slot < p.slots, c.status, kChkGlobalRow))
    p.ws_item[slot] = it.piece == 0 ? make_int4(pieces, r0 + tok0, toks, hk) : make_int4(0, 0, 0, 0);
  if (it.piece >= pieces) return;  // (the same for every warp)
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, L::TM_COLS);
    tmem_relinquish();
  }
  const int t0 = static_cast<int>(static_cast<long long>(all_a) * it.piece / pieces);
  const int a1 = static_cast<int>(static_cast<long long>(all_a) * (it.piece + 1) / pieces);
  const int n_a = a1 - t0;
  const int n_b = all_b == 0 ? 0 : (it.piece + 1 == pieces ? all_b : a1) - t0;
  const int n = max(n_a, n_b), both = min(n_a, n_b);
  auto first_key = [&](int t) { return keys.tile(t0 + t) * BN; };
  // V tiles [0, low) and [cut, n) are inspected: a window or the causal mask hides
  // some of their keys from some rows, or the sequence ends inside
  const int low = keys.lo_last > 0 ? max(0, min(n, keys.lo_last / BN + 1 - keys.skip - t0)) : 0;
  const int cut = max(low, min(n, max(0, it.past + tok0 + 1) / BN - keys.skip - t0));
  auto inspected = [&](int t) { return t < low || t >= cut; };
  auto inspected_before = [&](int t) { return t < low ? t : low + max(0, t - cut); };
  auto buffer_of = [&](int x, int t) {
    return NB <= 2 ? x : (t < both ? 2 * t + x : both + t) % NB;
  };
  auto bar_of = [&](int t) { return NB == 3 ? t % 3 : 0; };
  auto phase_of = [&](int t) { return NB == 3 ? t / 3 : t; };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return packed_warp_wait(bar, parity & 1, c.status, abort);
  };

  if (warp < 4) {
    if (kGather) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    auto load_q = [&](int x) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&ctrl->q_full[x], KCH * p.group * p.tok * 128);
        for (int ch = 0; ch < KCH; ++ch)
          tma_load_4d(smem + L::OFF_Q + x * L::Q_BYTES + ch * BM * 128, &maps.q, &ctrl->q_full[x],
                      ch * 64, hk * p.group, r0 + tok0 + x * p.tok, 0);
      }
    };
    if (warp == 0 && kGather) {
      load_q(0);
      if (n_b > 0) load_q(1);
      // (landed before the CTA can exit, whatever becomes of the others)
      const int zero = 0;
      mbar_wait(&ctrl->q_full[0], 0, &zero);
      if (n_b > 0) mbar_wait(&ctrl->q_full[1], 0, &zero);
    } else if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Lane l copies box l % boxes of chunk l / boxes of a tile.
      const int boxes = BN / p.box_rows;
      const int box = lane % boxes, chunk = lane / boxes;
      const bool mine = chunk < KCH;
      int page = c.pages, row = 0, next_page = c.pages, next_row = 0;
      bool next_missing = false;
      // (a lookup is used a tile later: its load is not waited for here)
      int raw = -1;
      bool looked = false;
      auto look_up = [&](int t) {
        looked = false;
        next_row = 0;
        if (t >= n || !mine) return;
        const int j = first_key(t) + box * p.box_rows;
        if (keys.unseen(j, p.box_rows)) return;
        if (j >= it.keys) return;
        looked = true;
        int entry;
        split_position(c, j, &entry, &next_row);
        raw = __ldg(c.table + it.b * c.table_stride + entry);
      };
      auto take = [&](int t) {  // the lookup of tile t becomes the current one
        next_missing = looked && (raw < 0 || raw >= c.pages);
        next_page = looked && !next_missing ? raw : c.pages;
        page = next_page, row = next_missing ? 0 : next_row;
        const bool any = __any_sync(0xffffffffu, next_missing);
        // (box by box: word w has keys 32 w ..)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t bits = 0u;
          if (any) {
            const int k0 = box * p.box_rows - 32 * w, k1 = k0 + p.box_rows;  // keys of this box
            if (next_missing && k1 > 0 && k0 < 32)
              bits = (0xFFFFFFFFu << max(k0, 0)) & (0xFFFFFFFFu >> (32 - min(k1, 32)));
            bits = __reduce_or_sync(0xffffffffu, bits);
          }
          if (lane == 0) *static_cast<volatile uint32_t*>(&ctrl->missing[t & 15][w]) = bits;
        }
        if (any && lane == 0) atomicOr(c.status, kStatusIndex);
        look_up(t + 1);
      };
      int k_fills = 0, v_fills = 0;
      auto load_kv = [&](int t, bool v) -> bool {
        const int s = t % NS;
        uint64_t* empty = v ? &ctrl->v_empty[s] : &ctrl->k_empty[s];
        uint64_t* full = v ? &ctrl->v_full[s] : &ctrl->k_full[s];
        if (!wait(empty, (t / NS) ^ 1)) return false;
        if (lane == 0) mbar_arrive_expect_tx(full, L::KV_BYTES);
        __syncwarp();
        uint8_t* dst = smem + (v ? L::OFF_V : L::OFF_K) + s * L::KV_BYTES;
        if (mine && JVP_CHECK(chunk * BN * 128 + (box + 1) * p.box_rows * 128 <= L::KV_BYTES, c.status,
                              kChkSmem))
          tma_load_4d(dst + chunk * BN * 128 + box * p.box_rows * 128, v ? &maps.v : &maps.k, full,
                      chunk * 64, row, hk, page);
        if (v && inspected(t) && lane == 0) mbar_arrive(&ctrl->v_issued[inspected_before(t) % NS]);
        ++(v ? v_fills : k_fills);
        return true;
      };
      load_q(0);
      look_up(0);
      take(0);
      bool ok = load_kv(0, false);
      if (n_b > 0) load_q(1);
      for (int t = 0; ok && t < n; ++t) {
        ok = load_kv(t, true);
        if (ok && t + 1 < n) {
          take(t + 1);
          ok = load_kv(t + 1, false);
        }
      }
      if (!ok) {
        // let every copy already issued land before the CTA can exit
        const int zero = 0;
        mbar_wait(&ctrl->q_full[0], 0, &zero);
        if (n_b > 0) mbar_wait(&ctrl->q_full[1], 0, &zero);
        for (int t = max(0, k_fills - NS); t < k_fills; ++t)
          mbar_wait(&ctrl->k_full[t % NS], (t / NS) & 1, &zero);
        for (int t = max(0, v_fills - NS); t < v_fills; ++t)
          mbar_wait(&ctrl->v_full[t % NS], (t / NS) & 1, &zero);
      }
    } else if (warp == 1 || (NB == 3 && warp == 2)) {
      // ---------------------------------------------------------- MMAs
      // (as in the packed kernel)
      const int w = warp - 1;
      const uint32_t neg_a = p.neg_scores ? (1u << 13) : 0u;
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::OFF_V), BN * 128, 1024);
      auto scores = [&](int x, int t, int buf, int bar) {
        const uint64_t qd = q_desc + x * (L::Q_BYTES >> 4);
        const uint64_t kd = k_desc + (t % NS) * (L::KV_BYTES >> 4);
#pragma unroll
        for (int ch = 0; ch < KCH; ++ch)
          mma_ss_x4_warp<2, 2>(tmem + L::TM_S + buf * BN, qd + ch * (BM * 128 / 16),
                               kd + ch * (BN * 128 / 16), IDESC_S | neg_a, ch > 0 ? 1u : 0u);
        mma_commit_warp(&ctrl->s_full[x][bar]);
      };
      auto k_landed = [&](int t) {
        const bool got = wait(&ctrl->k_full[t % NS], t / NS);
        tc_fence_after();
        return got;
      };
      auto v_landed = [&](int t) {
        const int k = inspected_before(t);
        return inspected(t) ? wait(&ctrl->v_checked[k % NS], k / NS)
                            : wait(&ctrl->v_full[t % NS], t / NS);
      };
      auto values = [&](int x, int t, int buf, int bar, int phase) {
        const uint64_t vd = v_desc + (t % NS) * (L::KV_BYTES >> 4);
        const uint32_t p_tm = tmem + L::TM_S + buf * BN, o_tm = tmem + L::TM_O + x * D;
        if (!wait(&ctrl->p_full[x][bar], phase)) return false;
        tc_fence_after();
        mma_ts_x4_warp<8, 128>(o_tm, p_tm, vd, IDESC_O, t > 0 ? 1u : 0u);
        mma_ts_x4_warp<8, 128>(o_tm, p_tm + 32, vd + 4 * 128, IDESC_O, 1u);
        return true;
      };
      bool ok = wait(&ctrl->q_full[0], 0) && k_landed(0);
      if (ok && w == 0) scores(0, 0, 0, 0);
      if (ok && n_b > 0) {
        ok = wait(&ctrl->q_full[1], 0);
        tc_fence_after();
        if (ok && w == 0) scores(1, 0, 1, 0);
      }
      if (ok) mma_commit_warp(&ctrl->k_empty[0]);
      if constexpr (NB <= 2) {
        for (int t = 0; ok && t < n; ++t) {
          const bool b_last = t < n_b;        // B is the last user of V(t) ...
          const bool b_last_k = t + 1 < n_b;  // ... and of K(t + 1)
          bool v_here = false, k_here = false;
#pragma unroll
          for (int x = 0; x < NQ; ++x) {
            const int nx = x ? n_b : n_a;
            if (!ok || t >= nx) continue;
            if (!v_here) ok = v_landed(t);
            v_here = true;
            if (!ok || !(ok = values(x, t, x, 0, t))) continue;
            if (b_last ? x == 1 : x == 0) mma_commit_warp(&ctrl->v_empty[t % NS]);
            if (t + 1 < nx) {
              if (!k_here && !(ok = k_landed(t + 1))) continue;
              k_here = true;
              scores(x, t + 1, x, 0);
              if (b_last_k ? x == 1 : x == 0) mma_commit_warp(&ctrl->k_empty[(t + 1) % NS]);
            } else {
              mma_commit_warp(&ctrl->o_full[x]);
            }
          }
        }
      } else {
        if (ok && both > 1) {  // A's scores against key tile 1: the third buffer
          if (w == 0) {
            ok = k_landed(1);
            if (ok) scores(0, 1, 2, 1);
          } else {
            mma_commit_warp(&ctrl->k_empty[1]);
          }
        }
        auto step = [&](int x, int t, int buf, int bar, int phase) {
          if (!(ok = v_landed(t) && values(x, t, buf, bar, phase))) return;
          mma_commit_warp(&ctrl->o_done[x][bar]);
          if (t + 1 == (x ? n_b : n_a)) mma_commit_warp(&ctrl->o_full[x]);
          mma_commit_warp(&ctrl->v_empty[t % NS]);
          const int ts = t + 1 + x;
          if (ts < both) {
            if (!(ok = k_landed(ts))) return;
            scores(1 - x, ts, buf, (bar + 1 + x) % 3);
            mma_commit_warp(&ctrl->k_empty[ts % NS]);
          }
        };
        for (int t = 0; ok && t < both; t += 3) {  // three key tiles are six steps
          const int ph = t / 3;
          if (w == 0) {
            step(0, t, 0, 0, ph);
            if (ok && t + 1 < both) step(0, t + 1, 2, 1, ph);
            if (ok && t + 2 < both) step(0, t + 2, 1, 2, ph);
          } else {
            step(1, t, 1, 0, ph);
            if (ok && t + 1 < both) step(1, t + 1, 0, 1, ph);
            if (ok && t + 2 < both) step(1, t + 2, 2, 2, ph);
          }
        }
        const int x = n_a > n_b ? 0 : 1;
        auto release = [&](uint64_t* bar) {  // for both warps
          mma_commit_warp(bar);
          mma_commit_warp(bar);
        };
        auto solo_scores = [&](int t) {
          if (t >= n || (t == 0 && both == 0)) return true;
          if (!k_landed(t)) return false;
          scores(x, t, (both + t) % NB, bar_of(t));
          release(&ctrl->k_empty[t % NS]);
          return true;
        };
        if (w == x) {
          if (ok && both < n) ok = solo_scores(both) && solo_scores(both + 1);
          for (int t = both; ok && t < n; ++t) {
            if (!(ok = v_landed(t) && values(x, t, (both + t) % NB, bar_of(t), phase_of(t)))) break;
            mma_commit_warp(&ctrl->o_done[x][bar_of(t)]);
            if (t + 1 == n) mma_commit_warp(&ctrl->o_full[x]);
            release(&ctrl->v_empty[t % NS]);
            ok = solo_scores(t + 2);
          }
        }
      }
      if (!ok) packed_timeout(c.status, abort);
      mma_commit_warp(&ctrl->drain[w]);
      const int zero = 0;
      mbar_wait(&ctrl->drain[w], 0, &zero);
    } else if (warp == 3) {
      // ---------------------------------------------------------- V inspector
      bool ok = true;
      for (int t = 0; ok && t < n; t = t + 1 < low || t + 1 >= cut ? t + 1 : cut) {
        if (!inspected(t)) continue;
        const int k = inspected_before(t);
        ok = wait(&ctrl->v_issued[k % NS], k / NS) && wait(&ctrl->v_full[t % NS], t / NS);
        if (!ok) break;
        const int j0 = first_key(t);
        const uint32_t v = smem_u32(smem + L::OFF_V + t % NS * L::KV_BYTES);
        const int rows = max(0, min(BN, it.keys - j0));
        for (int e = lane; e < (BN - rows) * KCH * 8; e += 32) {
          const int piece = e % 8, ch = (e / 8) % KCH, row = rows + e / (8 * KCH);
          if (JVP_CHECK(row < BN, c.status, kChkSmem))
            st_shared_v4(v + ch * BN * 128 + row * 128 + piece * 16, 0u, 0u, 0u, 0u);
        }
        // Rows that some token does not see: [0, hidden) and [from, rows).
        const int hidden = max(0, min(rows, keys.lo_last - j0));
        const int from = max(hidden, min(rows, max(0, it.past + tok0 + 1 - j0)));
        using E = PackedElem<T>;
        uint32_t seen[4] = {0u, 0u, 0u, 0u};
        for (int ch = 0; ch < KCH; ++ch) {
          const uint32_t base = v + ch * BN * 128;
#pragma unroll 4
          for (int e = lane; e < (hidden + rows - from) * 8; e += 32) {
            uint32_t x[4];
            ld_shared_v4(base + (e < hidden * 8 ? e : e + (from - hidden) * 8) * 16, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) E::zeros(x[i], &seen[i]);
          }
        }
        const uint32_t any = seen[0] | seen[1] | seen[2] | seen[3];
        if (__any_sync(0xffffffffu, (any & 0x7FFF7FFFu) != 0u)) {
          // infinities and NaN of the whole tile become zeros; rows that see them
          // add them at the end
          for (int e = lane; e < rows * 8 * KCH; e += 32) {
            const uint32_t at = v + (e / (rows * 8)) * BN * 128 + (e % (rows * 8)) * 16;
            uint32_t x[4];
            if (!JVP_CHECK(e % (rows * 8) * 16 + 16 <= BN * 128, c.status, kChkSmem)) continue;
            ld_shared_v4(at, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((x[i] & E::kExp) == E::kExp) x[i] &= 0xFFFF0000u;
              if ((x[i] >> 16 & E::kExp) == E::kExp) x[i] &= 0x0000FFFFu;
            }
            st_shared_v4(at, x[0], x[1], x[2], x[3]);
          }
          if (lane == 0)
            atomicOr(&ctrl->special, t < low ? 1 : 2);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->v_checked[k % NS]);
      }
    }
  } else if (kGather && warp < 8) {
    // ------------------------------------------------------------ gathering warps
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    using TC = typename std::conditional<SRC == kChunkE4M3, uint8_t, T>::type;
    constexpr int PR = D / 8, HP = PR / 2;  // pieces of a row; of a thread in half a tile
    constexpr int RS = 128 / PR;            // rows between a thread's pieces
    ChunkPlaces* const places = reinterpret_cast<ChunkPlaces*>(smem + L::OFF_PLACES);
    const int g = static_cast<int>(threadIdx.x) - 128;
    const int piece = g % PR, prow = g / PR;
    const bool in_row = piece * 8 < c.D;
    const TC* const kc = static_cast<const TC*>(c.k) + hk * c.sk.h + piece * 8;
    const TC* const vc = static_cast<const TC*>(c.v) + hk * c.sv.h + piece * 8;
    // where this thread's pieces of row r lie in a tile (rows differ by multiples of
    // 8 where RS is 8, so the swizzle is the same; RS = 16 too)
    const uint32_t in_tile = (piece / 8) * BN * 128 + prow * 128 + (((piece % 8) ^ (prow & 7)) << 4);
    const uint32_t stage = smem_u32(smem + L::OFF_STAGE) + g * 8;
    static_assert(RS % 8 == 0, "swizzle");
    // Key g of a tile: its block-table entry two tiles ahead, its scales one ahead.
    int raw = -1, raw_row = 0, page = -1, row = 0;
    bool looked = false, have = false, none = false;  // looked up; there; its page is not
    unsigned scales = 0;
    auto look_up = [&](int t) {  // the entry
      looked = false;
      if (t >= n) return;
      const int j = first_key(t) + g;
      if (keys.unseen(j, 1) || j >= it.keys) return;
      looked = true;
      int entry;
      split_position(c, j, &entry, &raw_row);
      raw = __ldg(c.table + it.b * c.table_stride + entry);
    };
    auto resolve = [&]() {  // the place, and its scales on their way
      have = looked && raw >= 0 && raw < c.pages;
      none = looked && !have;
      page = have ? raw : 0, row = have ? raw_row : 0;
      if (SRC == kChunkE4M3 && have) {
        const long long at = (static_cast<long long>(page) * c.Hkv + hk) * c.page_size + row;
        scales = __ldg(c.k_scale + at) | static_cast<unsigned>(__ldg(c.v_scale + at)) << 8;
      }
    };
    auto sync_gather = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    // The places of tile t for every thread, and the next tiles' lookups.
    auto publish = [&](int t) {
      sync_gather();  // the last tile's places have been read
      places->k[g] = have ? page * c.sk.b + row * c.sk.n : -1;
      places->v[g] = have ? page * c.sv.b + row * c.sv.n : -1;
      if (SRC == kChunkE4M3) {
        places->k_scale[t & 1][g] = static_cast<uint8_t>(have ? scales & 0xFFu : 127u);
        places->v_scale[t & 1][g] = static_cast<uint8_t>(have ? scales >> 8 : 127u);
      }
      const uint32_t gone = __ballot_sync(0xffffffffu, none);
      if (lane == 0) {
        *static_cast<volatile uint32_t*>(&ctrl->missing[t & 15][warp & 3]) = gone;
        if (gone) atomicOr(c.status, kStatusIndex);
      }
      resolve();
      look_up(t + 2);
      sync_gather();
    };
    // Half tile h: 4 t + 0, 1 of K's tile t, + 2, 3 of V's.
    bool ok = true;
    auto slot_of = [&](int t) { return t % NS; };
    auto wait_empty = [&](int t, bool v) {
      return wait(v ? &ctrl->v_empty[slot_of(t)] : &ctrl->k_empty[slot_of(t)], (t / NS) ^ 1);
    };
    auto issue = [&](int h) {
      const int t = h >> 2;
      // (whatever became of a wait: the warps meet here)
      if (t < n && (h & 3) == 0) publish(t);
      if (ok && t < n) {
        const bool v = (h & 2) != 0;
        const int r0h = (h & 1) * (BN / 2);
        if (SRC == kChunkRows && (h & 1) == 0) ok = wait_empty(t, v);
        if (ok) {
          const uint32_t tile = smem_u32(smem + (v ? L::OFF_V : L::OFF_K) + slot_of(t) * L::KV_BYTES);
          const uint32_t to = SRC == kChunkE4M3 ? stage + h % kChunkAhead * L::HALF_CODES
                                                : tile + in_tile + r0h * 128;
          const long long* at = v ? places->v : places->k;
          const TC* base = v ? vc : kc;
#pragma unroll
          for (int i = 0; i < HP; ++i) {
            const long long place = at[r0h + prow + i * RS];
            const bool on = in_row && place >= 0;
            if (!JVP_CHECK(r0h + prow + i * RS < BN, c.status, kChkSmem)) continue;
            if constexpr (SRC == kChunkE4M3)
              chunk_copy<8>(to + i * 128 * 8, base + (on ? place : 0), on);
            else
              chunk_copy<16>(to + i * RS * 128, base + (on ? place : 0), on);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(0);
    resolve();
    look_up(1);
    for (int h = 0; h < kChunkAhead; ++h) issue(h);
    for (int h = 0; h < 4 * n; ++h) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kChunkAhead - 1) : "memory");
      const int t = h >> 2;
      const bool v = (h & 2) != 0;
      if constexpr (SRC == kChunkE4M3) {
        if (ok && (h & 1) == 0) ok = wait_empty(t, v);
        if (ok) {
          const int r0h = (h & 1) * (BN / 2);
          const uint32_t from = stage + h % kChunkAhead * L::HALF_CODES;
          const uint32_t to = smem_u32(smem + (v ? L::OFF_V : L::OFF_K) + slot_of(t) * L::KV_BYTES) +
                              in_tile + r0h * 128;
          const uint8_t* scale = v ? places->v_scale[t & 1] : places->k_scale[t & 1];
#pragma unroll
          for (int i = 0; i < HP; ++i) {
            uint32_t w[2], y[4];
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(w[0]), "=r"(w[1])
                         : "r"(from + i * 128 * 8)
                         : "memory");
            const float f = scale_value(scale[r0h + prow + i * RS]);
            e4m3x4_to_half2x2(w[0], y[0], y[1]);
            e4m3x4_to_half2x2(w[1], y[2], y[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = chunk_decode<T>(y[k], f);
            st_shared_v4(to + i * RS * 128, y[0], y[1], y[2], y[3]);
          }
        }
      }
      // (the staging area's next half tile takes the place of the one just read)
      if (ok && v && (h & 1) == 0 && inspected(t) && g == 0)
        mbar_arrive(&ctrl->v_issued[inspected_before(t) % NS]);
      if (ok && (h & 1) == 1) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v ? &ctrl->v_full[slot_of(t)] : &ctrl->k_full[slot_of(t)]);
      }
      issue(h + kChunkAhead);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    // ------------------------------------------------------------ softmax
    if (kGather) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - kSoftmax) >> 2;  // query tile
    const int sub = warp & 3;       // its TMEM lanes 32 sub ..
    const int r = sub * 32 + lane;
    const int nx = x ? n_b : n_a;
    const int rt = r / p.group, rh = r - rt * p.group;  // token and head of the row
    const int first = tok0 + x * p.tok;                 // first token of the tile
    const int i = first + rt;                           // token within the sequence
    const bool row_ok = rt < p.tok && i < len;
    // The row sees keys [lo, limit) and the sinks; rows that are not used: all.
    const int at = it.past + i;  // its position
    const int limit = row_ok ? at + 1 : it.keys;
    const int lo = row_ok ? keys.lo(at) : 0;
    int warp_limit = limit, warp_lo = lo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      warp_limit = min(warp_limit, __shfl_xor_sync(0xffffffffu, warp_limit, o));
      warp_lo = max(warp_lo, __shfl_xor_sync(0xffffffffu, warp_lo, o));
    }
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t o_tm = lane_base + L::TM_O + x * D;
    const float scale = p.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;  // the base of the exponents, the sum
    bool ok = true;
    for (int t = 0; t < nx; ++t) {
      const uint32_t s_tm = lane_base + L::TM_S + buffer_of(x, t) * BN;
      if (!(ok = wait(&ctrl->s_full[x][bar_of(t)], phase_of(t)))) break;
      tc_fence_after();
      float s[BN];
      const bool s_cols = JVP_CHECK(buffer_of(x, t) < NB && buffer_of(x, t) >= 0, c.status, kChkTmem);
      if (!s_cols) continue;
#pragma unroll
      for (int q = 0; q < BN; q += 64) {
        uint32_t a[32], b[32];
        tmem_ld32x2(s_tm + q, s_tm + q + 32, a, b);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          s[q + e] = __uint_as_float(a[e]);
          s[q + 32 + e] = __uint_as_float(b[e]);
        }
      }
      const int j0 = first_key(t);
      if (j0 + BN > warp_limit) {
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (j0 + e >= limit) s[e] = -INFINITY;
      }
      if (j0 < warp_lo && j0 + BN > keys.sinks) {
        const int a = lo - j0, b = keys.sinks - j0;  // hidden: b <= e < a
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (e < a && e >= b) s[e] = -INFINITY;
      }
      uint32_t missing[4];
      ld_shared_v4(smem_u32(ctrl->missing[t & 15]), missing);
      if ((missing[0] | missing[1] | missing[2] | missing[3]) != 0u) {
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (missing[e / 32] & (1u << (e % 32))) s[e] = -INFINITY;
      }
      const float m_tile = packed_max(s) * scale;
      const bool need = m_tile - m_run > PackedElem<T>::kTop;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? packed_base<T>(m_tile) : m_run;
        const float alpha = need ? ex2_approx(m_run - m_new) : 1.f;
        l_run *= alpha;
        m_run = m_new;
        if (t > 0) {
          // (O has tile t - 1's product: see the packed kernel)
          if (NB == 3) {
            if (!(ok = wait(&ctrl->o_done[x][bar_of(t - 1)], phase_of(t - 1)))) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            if (!JVP_CHECK(L::TM_O + x * D + col + 32 <= L::TM_COLS, c.status, kChkTmem)) continue;
            uint32_t o[32];
            tmem_ld32(o_tm + col, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_tm + col, o);
          }
        }
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      const float2 c2 = make_float2(scale, scale), nm2 = make_float2(-m_use, -m_use);
      float2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int q = 0; q < BN; q += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 w = fma2(make_float2(s[q + e], s[q + e + 1]), c2, nm2);
          w.x = ex2_approx(w.x);
          w.y = ex2_approx(w.y);
          sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], w);
          pk[e >> 1] = PackedElem<T>::pack(w.x, w.y);
        }
        tmem_st16(s_tm + q / 2, pk);
      }
      l_run += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
               ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->p_full[x][bar_of(t)]);
    }
    // ------------------------------------------------------------ epilogue
    if (nx > 0 && ok && (ok = wait(&ctrl->o_full[x], 0))) {
      tc_fence_after();
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (NaN stays NaN)
      const bool in_t = JVP_CHECK(!row_ok || (r0 + i < p.T && hk * p.group + rh < p.H), c.status,
                                  kChkGlobalRow);
      const float lse2 = l_run == 0.f ? -INFINITY
                                      : m_run + PackedElem<T>::kShift +
                                            log2f(l_run * PackedElem<T>::kUnshift);
      const long long ws_row = (static_cast<long long>(slot) * NQ + x) * BM + r;
      if (row_ok && in_t) {
        if (slot >= 0) p.ws_lse[ws_row] = lse2;
        else if (p.lse)
          p.lse[static_cast<long long>(hk * p.group + rh) * p.T + r0 + i] = lse2 * 0.6931471805599453f;
      }
      // A whole tile of tokens: through the (now idle) Q tile, 16-byte piece k of
      // row r at position k ^ (r % 8), and a TMA store of the box.  Else the
      // sequence ends inside the tile, and each thread writes its row; of a piece,
      // in fp32 to the workspace.
      const bool whole = slot < 0 && first + p.tok <= len;
      const int special = *static_cast<volatile int*>(&ctrl->special);
      const uint32_t stage = smem_u32(smem + L::OFF_Q + x * L::Q_BYTES) + r * 128;
      T* dst = static_cast<T*>(p.o) + static_cast<long long>(r0 + i) * p.so.n +
               static_cast<long long>(hk * p.group + rh) * p.so.h;
      // Sums of the infinities and NaN in columns d .. d + 7 of the values that the
      // row sees among the tiles set apart (weights are positive: infinities keep
      // their sign).
      auto add_special = [&](int d, float (&y)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = 0.f;
        if (d >= c.D) return;
#pragma unroll 1
        for (int t = 0; t < nx; ++t) {
          if (!inspected(t) || !(special & (t < low ? 1 : 2))) continue;
          const int j1 = min(first_key(t) + BN, it.keys);
#pragma unroll 1
          for (int j = first_key(t); j < j1; ++j) {
            if (!keys.sees(at, j)) continue;
            int entry, in_page;
            split_position(c, j, &entry, &in_page);
            const int page = page_of(c, it.b, entry);
            if (page < 0) continue;
            const long long place = page * c.sv.b + hk * c.sv.h + in_page * c.sv.n + d;
            uint32_t w[4];
            if constexpr (SRC == kChunkE4M3) {
              const uint2 codes =
                  __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + place));
              const float f = scale_value(__ldg(
                  c.v_scale + (static_cast<long long>(page) * c.Hkv + hk) * c.page_size + in_page));
              e4m3x4_to_half2x2(codes.x, w[0], w[1]);
              e4m3x4_to_half2x2(codes.y, w[2], w[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = chunk_decode<T>(w[k], f);
            } else {
              const uint4 x4 =
                  __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(c.v) + place));
              w[0] = x4.x, w[1] = x4.y, w[2] = x4.z, w[3] = x4.w;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t bits = w[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
              if ((bits & PackedElem<T>::kExp) == PackedElem<T>::kExp) y[k] += PackedElem<T>::get(bits);
            }
          }
        }
      };
#pragma unroll
      for (int col = 0; col < D; col += 64) {
        uint32_t o[2][32];
        tmem_ld32x2(o_tm + col, o_tm + col + 32, o[0], o[1]);
        if (special && row_ok) {
#pragma unroll
          for (int e = 0; e < 64; e += 8) {
            float y[8];
            add_special(col + e, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t& to = o[(e + k) / 32][(e + k) % 32];
              to = __float_as_uint(__uint_as_float(to) + y[k]);
            }
          }
        }
        if (slot >= 0) {
          if (row_ok && JVP_CHECK(slot < p.slots, c.status, kChkGlobalRow)) {
            float4* to = reinterpret_cast<float4*>(p.ws_o + ws_row * D + col);
#pragma unroll
            for (int e = 0; e < 64; e += 4)
              to[e / 4] = make_float4(__uint_as_float(o[e / 32][e % 32]) * inv,
                                      __uint_as_float(o[e / 32][e % 32 + 1]) * inv,
                                      __uint_as_float(o[e / 32][e % 32 + 2]) * inv,
                                      __uint_as_float(o[e / 32][e % 32 + 3]) * inv);
          }
          continue;
        }
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = PackedElem<T>::pack(__uint_as_float(o[e / 32][e % 32 + 2 * k]) * inv,
                                       __uint_as_float(o[e / 32][e % 32 + 2 * k + 1]) * inv);
          if (!JVP_CHECK((col / 64) * BM * 128 + r * 128 + 128 <= L::Q_BYTES, c.status, kChkSmem))
            continue;
          if (whole)
            st_shared_v4(stage + (col / 64) * BM * 128 + (((e / 8) ^ (r & 7)) << 4), w[0], w[1],
                         w[2], w[3]);
          else if (row_ok && in_t && col + e < c.D &&
                   JVP_CHECK(col + e + 8 <= c.D, c.status, kChkGlobalCol))
            *reinterpret_cast<uint4*>(dst + col + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (whole) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->staged[x]);
        if (warp == kSoftmax + 4 * x && wait(&ctrl->staged[x], 0) && lane == 0) {
          for (int ch = 0; ch < KCH; ++ch)
            tma_store_4d(&maps.o, smem + L::OFF_Q + x * L::Q_BYTES + ch * BM * 128, ch * 64,
                         hk * p.group, r0 + first, 0);
          tma_store_commit();
          tma_store_wait_read();  // shared memory stays valid until then
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TM_COLS);
  }
}

template <typename T, int D, int NQ, ChunkSource SRC>
cudaError_t launch_chunk_tc_variant(const ChunkMaps& maps, const ChunkParams& p,
                                    cudaStream_t stream) {
  constexpr int smem = ChunkLayout<D, NQ, SRC>::BYTES;
  const cudaError_t e = allow_shared_memory<chunk_tc_kernel<T, D, NQ, SRC>>(smem);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.units) * p.heads;
  chunk_tc_kernel<T, D, NQ, SRC>
      <<<static_cast<unsigned>(grid), chunk_threads(NQ, SRC), smem, stream>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace jvp
