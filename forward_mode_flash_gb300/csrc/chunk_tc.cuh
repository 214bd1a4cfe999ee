// chunk_tc.cuh -- attention of chunks of new tokens over a paged cache on the
// tensor cores (tcgen05 + TMEM), fp16 / bf16, fp32 accumulation.
//
// The softmax, its rounding and the flow between copies, products and softmax are
// those of the kernel over packed prompts (packed_tc.cuh): 128-row query tiles of
// `tok` tokens times the query heads of a key/value head, two tiles (NQ) per CTA
// against the same ring of 128-key K/V tiles.  What differs:
//   - Key tiles are collected from pages.  SRC = kChunkBoxes: the largest power of
//     two of rows that divides a page (8 at least) is one TMA box; the lanes of two
//     copying warps, one for Q and K, one for V, each look up one box's page a tile ahead
//     and issue its copy.  A box that no row sees, or whose page does not exist, is copied
//     from behind the last page, where TMA writes zeros.
//     The other sources have eight gathering warps, two for each half of a tile's keys or
//     values, a lane looking up a row two tiles ahead.  kChunkRows (16-bit pages of any
//     size): asynchronous 16-byte copies straight into the tile.  kChunkStaged (e4m3,
//     pages of 8-row boxes): TMA copies boxes of codes to a staging ring several half tiles
//     ahead, and the warps convert them.  kChunkE4M3 (other pages): the warps copy the codes
//     themselves, in 8-byte pieces.  A code is exact in fp16 and bf16; times its scale, it
//     is rounded to T as cache_read does.
//   - A row sees an interval of keys and the sinks (ChunkKeys); tiles that no row
//     sees are left out.  What is hidden is one word of bits per 32 keys.
//   - A CTA takes an equal part of all work, whatever the lengths (chunk.cuh), its items
//     one behind the other: copies and products of the next go on behind the last one's
//     epilogue.  One warp finds the parts and puts them into shared memory for the others,
//     and inspects those V tiles of which some rows see only a part.  Parts of cut items
//     are joined by another kernel in a fixed order.
// Keys of pages that do not exist are masked by a bit each.
//
// Bound: at D = 128 a pair of query tiles takes 1.55 us a key tile from boxes, 2.0 us
// from rows, 2.25 us from codes (1.27 us is the tensor core's at its measured rate,
// and the exponentials alone 1.07 us); at D = 64 1.4, 1.87 and 1.93 us.  A call begins and
// ends with some 20 us that no tile hides: 3.7 us until a CTA knows its part, 4 to 6 us to its
// first scores, 2.5 us of epilogue, 5 us for the join: most of it first passes over
// instructions.
#pragma once

#include "chunk.cuh"
#include "packed_tc.cuh"

namespace jvp {

// The gathering sources: 640 threads of 96 registers at launch (copies and products 80, two
// warpgroups of gathering 64 each, two of softmax 136: 480 = 5 * 96); their staging area lies
// behind the control block.
constexpr int kGatherWarps = 8;
constexpr int chunk_threads(int NQ, ChunkSource src) {
  return packed_threads(NQ) + (src == kChunkBoxes ? 0 : 32 * kGatherWarps);
}
// Half tiles of codes in flight by TMA: what the shared memory left holds.
constexpr int chunk_ahead(int D) { return D > 64 ? 4 : 8; }
template <int D, int NQ, ChunkSource SRC>
struct ChunkLayout : PackedLayout<D, NQ> {
  using P = PackedLayout<D, NQ>;
  static constexpr int AHEAD = chunk_ahead(D);
  static constexpr int NB = NQ;  // score buffers: one for each query tile
  static constexpr uint32_t TM_O = NB * P::BN;
  static_assert(NB * P::BN + NQ * D <= P::TM_COLS, "TMEM columns");
  static constexpr int HALF_CODES = 64 * D;  // bytes of half a tile of codes
  static constexpr int CTRL = 2048;  // control block
  static constexpr int OFF_STAGE = P::OFF_CTRL + CTRL;
  // (and 1024 for alignment)
  static constexpr int BYTES = OFF_STAGE + 1024 + (SRC == kChunkE4M3 || SRC == kChunkStaged ? AHEAD * HALF_CODES : 0);
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
  static_assert(SRC != kChunkBoxes || (3 - NQ) * (BYTES + 1024) <= 228 * 1024, "CTAs per SM");
};

// A CTA's part as its roles see it: key tiles of the query tiles (n: the larger; 0: no
// more parts); V tiles [0, low) and [cut, n) are inspected.
struct ChunkJob : ChunkPart<kChunkTile> {
  int n_a, n_b, n, low, cut;
  __device__ __forceinline__ void shape(const ChunkParams& p) {
    // A's key tiles are cut; where B has more they go with the last part
    const int all_b = toks > p.tok ? see.tiles(past + tok0 + toks - 1) : 0;
    n_a = t1 - t0;
    n_b = all_b == 0 ? 0 : (t1 == all ? all_b : t1) - t0;
    n = max(n_a, n_b);
    // a window or the causal mask hides some of their keys from some rows, or the
    // sequence ends inside
    low = see.lo_last > 0 ? max(0, min(n, see.lo_last / kChunkTile + 1 - see.skip - t0)) : 0;
    cut = max(low, min(n, max(0, past + tok0 + 1) / kChunkTile - see.skip - t0));
  }
  __device__ __forceinline__ bool inspected(int t) const { return t < low || t >= cut; }
  // inspected tiles before tile t
  __device__ __forceinline__ int before(int t) const { return t < low ? t : low + max(0, t - cut); }
  __device__ __forceinline__ int first_key(int t) const { return see.tile(t0 + t) * kChunkTile; }
};
constexpr int kChunkJobs = 4;  // parts in shared memory

template <int NS, int AHEAD>
struct ChunkCtrl {
  uint64_t q_full[2];
  uint64_t done[2];  // a part's epilogue of the query tile has ended
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t v_issued[NS], v_checked[NS];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t staged[2];
  uint64_t drain;
  uint64_t stage_full[AHEAD], stage_empty[AHEAD];  // half tiles of codes
  // Parts, written by one warp and read by the others, which hold little else of them
  // in registers: what spills goes through an L1 of the 28 KB that shared memory leaves.
  uint64_t job_full[kChunkJobs], job_empty[kChunkJobs];
  ChunkJob job[kChunkJobs];
  // By key tile modulo 8 (lookups are at most NS + 1 tiles ahead of the softmax), a bit
  // for every key: its page does not exist.
  alignas(16) uint32_t missing[8][4];
  // By part modulo 8 (copies are at most NS parts ahead): the number of the part,
  // counted from 1, if V entries were infinite or NaN where the window ([0]) or the
  // causal mask ([1]) cuts a tile.
  int special[8][2];
  uint32_t tmem_base;
  int abort;
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
  constexpr int BM = L::BM, BN = L::BN, NS = L::NS, KCH = L::KCH;
  constexpr int THREADS = chunk_threads(NQ, SRC);
  constexpr bool kGather = SRC != kChunkBoxes;
  constexpr bool kCodes = SRC == kChunkE4M3 || SRC == kChunkStaged;
  constexpr int kSoftmax = kGather ? 4 + kGatherWarps : 4;  // first softmax warp
  constexpr bool kBF16 = PackedElem<T>::kBF16;
  constexpr uint32_t IDESC_S = idesc_f16(kBF16, BM, BN, false);
  constexpr uint32_t IDESC_O = idesc_f16(kBF16, BM, D, true);
  static_assert(BN == kChunkTile, "key tiles");

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using Ctrl = ChunkCtrl<NS, L::AHEAD>;
  static_assert(sizeof(Ctrl) <= L::CTRL && NS <= 6, "control block budget");
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + L::OFF_CTRL);
  volatile int* abort = &ctrl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedCache& c = p.c;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.o);
      if (p.box_rows > 0) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&ctrl->q_full[x], 1);
        mbar_init(&ctrl->done[x], 4);  // one arrival per softmax warp of the tile
        mbar_init(&ctrl->s_full[x], 1);
        mbar_init(&ctrl->p_full[x], 4);
        mbar_init(&ctrl->o_full[x], 1);
        mbar_init(&ctrl->staged[x], 4);
      }
      mbar_init(&ctrl->drain, 1);
      for (int s = 0; s < NS; ++s) {
        mbar_init(&ctrl->k_full[s], kGather ? kGatherWarps / 2 : 1);
        mbar_init(&ctrl->k_empty[s], 1);
        mbar_init(&ctrl->v_full[s], kGather ? kGatherWarps / 2 : 1);
        mbar_init(&ctrl->v_empty[s], 1);
        mbar_init(&ctrl->v_issued[s], 1);
        mbar_init(&ctrl->v_checked[s], 1);
      }
      for (int s = 0; s < kChunkJobs; ++s) {
        mbar_init(&ctrl->job_full[s], 1);
        // a warp each: copies, products, inspection, softmax, gathering
        mbar_init(&ctrl->job_empty[s], 4 + 4 * NQ + (kGather ? kGatherWarps : 0));
      }
      for (int s = 0; s < L::AHEAD; ++s) {
        mbar_init(&ctrl->stage_full[s], 1);
        mbar_init(&ctrl->stage_empty[s], 2);
      }
      ctrl->abort = 0;
      fence_barrier_init();
    }
    if (lane < 16) (&ctrl->special[0][0])[lane] = 0;
  }
  ChunkSpan span;
  static_assert(sizeof(ChunkScratch) <= L::OFF_CTRL - L::OFF_K, "the tiles' space");
  if (!chunk_divide<BN, THREADS>(p, reinterpret_cast<ChunkScratch*>(smem + L::OFF_K), &span))
    return;
  fence_proxy_async_smem();  // TMA writes tiles where the division's scratch was
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, L::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // (as packed_warp_wait)
    const bool got = mbar_wait<false>(bar, parity & 1, abort);
    if (!got) packed_timeout(c.status, abort);
    return __all_sync(0xffffffffu, got);
  };
  // One warp walks the CTA's parts; the others take them from shared memory.  Barriers
  // go on from part to part, so each role counts what came before: `base` key tiles,
  // `seen` inspected V tiles, `uses` of each query tile and, in `steps`, its key tiles.
  auto take_job = [&](int k) -> const ChunkJob* {  // nullptr: there is none
    if (!wait(&ctrl->job_full[k % kChunkJobs], k / kChunkJobs)) return nullptr;
    const ChunkJob* j = &ctrl->job[k % kChunkJobs];
    return *static_cast<const volatile int*>(&j->n) > 0 ? j : nullptr;
  };
  auto leave_job = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctrl->job_empty[k % kChunkJobs]);
  };

  if (warp < 4) {
    if (kGather) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- copies
      // Warp 0 copies query tiles and K, warp 2 V (a copy's issue takes some 40 cycles, and
      // pages of 16 rows need 32 of them for a tile of K at D = 128; one warp for both: 1.8
      // to 1.9 us a tile, 1.5 with pages of 64).  Boxes: lane l copies box l % boxes of
      // chunk l / boxes of a tile.  Of codes (one chunk) warp 0 copies K and V to the
      // staging area, half a tile at a time.
      const bool values = warp == 2;
      const bool copies = SRC == kChunkBoxes || (SRC == kChunkStaged && !values);
      const int boxes = copies ? BN / p.box_rows : 1;
      const int box = lane % boxes, chunk = lane / boxes;
      const bool mine = copies && chunk < (kGather ? 1 : KCH);
      int base = 0, seen = 0, halves = 0;
      int uses[2] = {0, 0};
      int fills = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const ChunkJob* const job = take_job(k);
        if (!job) break;
        const ChunkJob &w = *job, &g = *job;
        auto load_q = [&](int x) -> bool {
          if (uses[x] > 0 && !wait(&ctrl->done[x], uses[x] - 1)) return false;
          ++uses[x];
          if (lane == 0) {
            mbar_arrive_expect_tx(&ctrl->q_full[x], KCH * p.group * p.tok * 128);
            for (int ch = 0; ch < KCH; ++ch)
              tma_load_4d(smem + L::OFF_Q + x * L::Q_BYTES + ch * BM * 128, &maps.q,
                          &ctrl->q_full[x], ch * 64, w.head * p.group,
                          w.r0 + w.tok0 + x * p.tok, 0);
          }
          return true;
        };
        // A lookup is used a tile later: its load is not waited for at once.
        int page = c.pages, row = 0, raw = -1, raw_row = 0;
        bool looked = false;
        auto look_up = [&](int t) {
          looked = false;
          if (t >= g.n || !mine) return;
          const int j = g.first_key(t) + box * p.box_rows;
          if (w.see.unseen(j, p.box_rows) || j >= w.keys) return;
          looked = true;
          int entry;
          split_position(c, j, &entry, &raw_row);
          raw = __ldg(c.table + w.b * c.table_stride + entry);
        };
        auto take = [&](int t) {  // the lookup of tile t becomes the current one
          const bool none = looked && (raw < 0 || raw >= c.pages);
          const bool have = looked && !none;
          page = have ? raw : c.pages, row = have ? raw_row : 0;
          if (!kGather && !values) {
            const bool any = __any_sync(0xffffffffu, none);
            // (box by box: word i has keys 32 i ..)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t bits = 0u;
              if (any) {
                const int k0 = box * p.box_rows - 32 * i, k1 = k0 + p.box_rows;
                if (none && k1 > 0 && k0 < 32)
                  bits = (0xFFFFFFFFu << max(k0, 0)) & (0xFFFFFFFFu >> (32 - min(k1, 32)));
                bits = __reduce_or_sync(0xffffffffu, bits);
              }
              if (lane == 0)
                *static_cast<volatile uint32_t*>(&ctrl->missing[(base + t) & 7][i]) = bits;
            }
            if (any && lane == 0) atomicOr(c.status, kStatusIndex);
          }
          look_up(t + 1);
        };
        auto load_kv = [&](int t, bool v) -> bool {
          if constexpr (SRC == kChunkStaged) {
            for (int i = 0; i < 2; ++i) {
              const int s = halves % L::AHEAD;
              if (!wait(&ctrl->stage_empty[s], (halves / L::AHEAD) ^ 1)) return false;
              if (lane == 0) mbar_arrive_expect_tx(&ctrl->stage_full[s], L::HALF_CODES);
              __syncwarp();
              const int b0 = box - i * boxes / 2;  // box of this half
              if (mine && b0 >= 0 && b0 < boxes / 2)
                tma_load_4d(smem + L::OFF_STAGE + s * L::HALF_CODES + b0 * p.box_rows * D,
                            v ? &maps.v : &maps.k, &ctrl->stage_full[s], 0, row, w.head, page);
              ++halves;
            }
            return true;
          } else {
            const int s = (base + t) % NS;
            uint64_t* empty = v ? &ctrl->v_empty[s] : &ctrl->k_empty[s];
            uint64_t* full = v ? &ctrl->v_full[s] : &ctrl->k_full[s];
            if (!wait(empty, ((base + t) / NS) ^ 1)) return false;
            if (lane == 0) mbar_arrive_expect_tx(full, L::KV_BYTES);
            __syncwarp();
            uint8_t* dst = smem + (v ? L::OFF_V : L::OFF_K) + s * L::KV_BYTES;
            if (mine && JVP_CHECK(chunk * BN * 128 + (box + 1) * p.box_rows * 128 <= L::KV_BYTES,
                                  c.status, kChkSmem))
              tma_load_4d(dst + chunk * BN * 128 + box * p.box_rows * 128, v ? &maps.v : &maps.k,
                          full, chunk * 64, row, w.head, page);
            if (v && g.inspected(t) && lane == 0)
              mbar_arrive(&ctrl->v_issued[(seen + g.before(t)) % NS]);
            ++fills;
            return true;
          }
        };
        if (copies) {
          look_up(0);
          take(0);
        }
        // (the first copy of the next part does not wait for this one's epilogues)
        if (!values && base == 0) ok = load_q(0) && (g.n_b == 0 || load_q(1));
        if (ok && copies) ok = load_kv(0, values) && (!kGather || load_kv(0, true));
        if (ok && !values && base > 0) ok = load_q(0) && (g.n_b == 0 || load_q(1));
        for (int t = 1; ok && copies && t < g.n; ++t) {
          take(t);
          ok = load_kv(t, values) && (!kGather || load_kv(t, true));
        }
        base += g.n, seen += g.before(g.n);
        leave_job(k);
      }
      // Every copy issued lands before the CTA can exit.
      const int zero = 0;
      for (int x = 0; x < 2; ++x)
        if (uses[x] > 0) mbar_wait(&ctrl->q_full[x], (uses[x] - 1) & 1, &zero);
      if (!ok) {
        for (int t = max(0, fills - NS); t < fills; ++t)
          mbar_wait(values ? &ctrl->v_full[t % NS] : &ctrl->k_full[t % NS], (t / NS) & 1, &zero);
        for (int h = max(0, halves - L::AHEAD); h < halves; ++h)
          mbar_wait(&ctrl->stage_full[h % L::AHEAD], (h / L::AHEAD) & 1, &zero);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMAs
      // (as in the packed kernel)
      const uint32_t neg_a = p.neg_scores ? (1u << 13) : 0u;
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::OFF_V), BN * 128, 1024);
      int base = 0, seen = 0;
      int uses[2] = {0, 0};
      int steps[2] = {0, 0};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const ChunkJob* const job = take_job(k);
        if (!job) break;
        const ChunkJob& g = *job;
        const int n_a = g.n_a, n_b = g.n_b, n = g.n;
        auto scores = [&](int x, int t) {
          const uint64_t qd = q_desc + x * (L::Q_BYTES >> 4);
          const uint64_t kd = k_desc + ((base + t) % NS) * (L::KV_BYTES >> 4);
#pragma unroll
          for (int ch = 0; ch < KCH; ++ch)
            mma_ss_x4_warp<2, 2>(tmem + L::TM_S + x * BN, qd + ch * (BM * 128 / 16),
                                 kd + ch * (BN * 128 / 16), IDESC_S | neg_a, ch > 0 ? 1u : 0u);
          mma_commit_warp(&ctrl->s_full[x]);
        };
        auto k_landed = [&](int t) {
          const bool got = wait(&ctrl->k_full[(base + t) % NS], (base + t) / NS);
          tc_fence_after();
          return got;
        };
        auto v_landed = [&](int t) {
          const int k = seen + g.before(t);
          return g.inspected(t) ? wait(&ctrl->v_checked[k % NS], k / NS)
                                : wait(&ctrl->v_full[(base + t) % NS], (base + t) / NS);
        };
        // (the tensor core runs this warp's products in order: scores issued behind a
        // product may overwrite its weights)
        auto values = [&](int x, int t) {
          const uint64_t vd = v_desc + ((base + t) % NS) * (L::KV_BYTES >> 4);
          const uint32_t p_tm = tmem + L::TM_S + x * BN, o_tm = tmem + L::TM_O + x * D;
          if (!wait(&ctrl->p_full[x], steps[x] + t)) return false;
          tc_fence_after();
          mma_ts_x4_warp<8, 128>(o_tm, p_tm, vd, IDESC_O, t > 0 ? 1u : 0u);
          mma_ts_x4_warp<8, 128>(o_tm, p_tm + 32, vd + 4 * 128, IDESC_O, 1u);
          return true;
        };
        auto free_k = [&](int t) { mma_commit_warp(&ctrl->k_empty[(base + t) % NS]); };
        auto free_v = [&](int t) { mma_commit_warp(&ctrl->v_empty[(base + t) % NS]); };
        // (O is free: the query tile was copied behind the epilogue of the part before)
        ok = wait(&ctrl->q_full[0], uses[0]) && k_landed(0);
        if (ok) scores(0, 0);
        if (ok && n_b > 0) {
          ok = wait(&ctrl->q_full[1], uses[1]);
          tc_fence_after();
          if (ok) scores(1, 0);
        }
        if (ok) free_k(0);
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
            if (!ok || !(ok = values(x, t))) continue;
            if (b_last ? x == 1 : x == 0) free_v(t);
            if (t + 1 < nx) {
              if (!k_here && !(ok = k_landed(t + 1))) continue;
              k_here = true;
              scores(x, t + 1);
              if (b_last_k ? x == 1 : x == 0) free_k(t + 1);
            } else {
              mma_commit_warp(&ctrl->o_full[x]);
            }
          }
        }
        base += n, seen += g.before(n);
        steps[0] += n_a, steps[1] += n_b;
        ++uses[0], uses[1] += n_b > 0;
        leave_job(k);
      }
      if (!ok) packed_timeout(c.status, abort);
      mma_commit_warp(&ctrl->drain);
      const int zero = 0;
      mbar_wait(&ctrl->drain, 0, &zero);
    } else if (warp == 3) {
      // ---------------------------------------------------------- the parts, V's inspection
      ChunkWalk<BN> walk(p, span.start, span.end);
      bool more = true;
      auto publish = [&](int k) {  // part k for all, n = 0 behind the last
        if (!more) return true;
        ChunkJob job;
        more = walk.next(p, &job);
        if (more) job.shape(p);
        else job.n = 0;
        if (!wait(&ctrl->job_empty[k % kChunkJobs], (k / kChunkJobs) ^ 1)) return false;
        if (lane == 0) {
          ctrl->job[k % kChunkJobs] = job;
          mbar_arrive(&ctrl->job_full[k % kChunkJobs]);
        }
        return true;
      };
      int base = 0, seen = 0, number = 0;
      bool ok = publish(0) && publish(1);
      for (int job_k = 0; ok; ++job_k) {
        if (!(ok = publish(job_k + 2))) break;
        const ChunkJob* const job = take_job(job_k);
        if (!job) break;
        const ChunkJob &w = *job, &g = *job;
        ++number;
        for (int t = g.low > 0 ? 0 : g.cut; ok && t < g.n; t = t + 1 < g.low ? t + 1 : max(t + 1, g.cut)) {
          const int k = seen + g.before(t), s = (base + t) % NS;
          ok = wait(&ctrl->v_issued[k % NS], k / NS) && wait(&ctrl->v_full[s], (base + t) / NS);
          if (!ok) break;
          const int j0 = g.first_key(t);
          const uint32_t v = smem_u32(smem + L::OFF_V + s * L::KV_BYTES);
          const int rows = max(0, min(BN, w.keys - j0));
          for (int e = lane; e < (BN - rows) * KCH * 8; e += 32) {
            const int piece = e % 8, ch = (e / 8) % KCH, row = rows + e / (8 * KCH);
            if (JVP_CHECK(row < BN, c.status, kChkSmem))
              st_shared_v4(v + ch * BN * 128 + row * 128 + piece * 16, 0u, 0u, 0u, 0u);
          }
          // Rows that some token does not see: [0, hidden) and [from, rows).
          const int hidden = max(0, min(rows, w.see.lo_last - j0));
          const int from = max(hidden, min(rows, max(0, w.past + w.tok0 + 1 - j0)));
          using E = PackedElem<T>;
          uint32_t found[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int part = 0; part < 2 * KCH; ++part) {
            const uint32_t at = v + (part >> 1) * BN * 128;
            const uint32_t last = at + (part & 1 ? rows : hidden) * 128;
#pragma unroll 4
            for (uint32_t to = at + (part & 1 ? from : 0) * 128 + lane * 16; to < last; to += 512) {
              uint32_t x[4];
              ld_shared_v4(to, x);
#pragma unroll
              for (int i = 0; i < 4; ++i) E::zeros(x[i], &found[i]);
            }
          }
          const uint32_t any = found[0] | found[1] | found[2] | found[3];
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
              *static_cast<volatile int*>(&ctrl->special[number & 7][t < g.low ? 0 : 1]) = number;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->v_checked[k % NS]);
        }
        base += g.n, seen += g.before(g.n);
        leave_job(job_k);
      }
    }
  } else if (kGather && warp < kSoftmax) {
    // ------------------------------------------------------------ gathering warps
    // Two warps for each half of a tile's keys or values, so that each has one half to
    // wait for, fill and hand on in a tile: 32 rows, of which lane l looks up row l (its
    // block-table entry two tiles ahead, its scale one ahead).  A row's 8-element pieces
    // are PR lanes', RI rows at once.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    using TC = typename std::conditional<kCodes, uint8_t, T>::type;
    constexpr int PR = D / 8, RI = 32 / PR, HP = 32 / RI;
    static_assert(kGatherWarps == 8 && L::AHEAD % 4 == 0, "two warps a half");
    const int gw = warp - 4, quarter = gw >> 1, piece = lane % PR, sub = lane / PR;
    const bool v = quarter >= 2, in_row = piece * 8 < c.D;
    const int row0 = (quarter & 1) * (BN / 2) + (gw & 1) * 32;  // of the tile
    uint64_t* const full = v ? ctrl->v_full : ctrl->k_full;
    uint64_t* const empty = v ? ctrl->v_empty : ctrl->k_empty;
    const Strides& stride = v ? c.sv : c.sk;
    const uint8_t* const scales = v ? c.v_scale : c.k_scale;
    const uint32_t ring = smem_u32(smem + (v ? L::OFF_V : L::OFF_K)) + (piece / 8) * BN * 128 +
                          (row0 + sub) * 128;
    // piece i of this lane (16 bytes, swizzled by the row modulo 8)
    auto tile_at = [&](int i) { return RI * i * 128 + (((piece % 8) ^ ((sub + RI * i) & 7)) << 4); };
    const uint32_t stage = smem_u32(smem + L::OFF_STAGE) + ((gw & 1) * 32 + sub) * D + piece * 8;
    int base = 0, seen = 0;
    bool ok = true;
    for (int job_k = 0; ok; ++job_k) {
      const ChunkJob* const job = take_job(job_k);
      if (!job) break;
      const ChunkJob &w = *job, &g = *job;
      const int n = g.n;
      const TC* const rows = static_cast<const TC*>(v ? c.v : c.k) + w.head * stride.h + piece * 8;
      int raw = -1, raw_row = 0, page = 0, row = 0;
      bool looked = false, have = false, none = false;  // looked up; there; its page is not
      unsigned next_scale = 127, scale = 127;
      long long place = -1;  // of the current tile, in elements from the start of the cache
      auto look_up = [&](int t) {  // the entry
        looked = false;
        if (t >= n) return;
        const int j = g.first_key(t) + row0 + lane;
        if (w.see.unseen(j, 1) || j >= w.keys) return;
        looked = true;
        int entry;
        split_position(c, j, &entry, &raw_row);
        raw = __ldg(c.table + w.b * c.table_stride + entry);
      };
      auto resolve = [&]() {  // the place, and its scale on its way
        have = looked && raw >= 0 && raw < c.pages;
        none = looked && !have;
        page = have ? raw : 0, row = have ? raw_row : 0;
        if (kCodes) {
          next_scale = 127;
          if (have)
            next_scale = __ldg(scales + (static_cast<long long>(page) * c.Hkv + w.head) * c.page_size +
                               row);
        }
      };
      auto take = [&](int t) {  // tile t becomes the current one; the next tiles' lookups
        if (SRC != kChunkStaged) place = have ? page * stride.b + row * stride.n : -1;
        scale = next_scale;
        const uint32_t gone = __ballot_sync(0xffffffffu, none);
        if (!v && lane == 0) {
          *static_cast<volatile uint32_t*>(&ctrl->missing[(base + t) & 7][row0 / 32]) = gone;
          if (gone) atomicOr(c.status, kStatusIndex);
        }
        resolve();
        look_up(t + 2);
      };
      auto wait_empty = [&](int t) {
        return wait(&empty[(base + t) % NS], ((base + t) / NS) ^ 1);
      };
      // Starts the copies of tile t, to its place or (codes) to the staging area.
      auto issue = [&](int t) {
        if (ok && t < n) {
          take(t);
          if (SRC == kChunkRows) ok = wait_empty(t);
          const uint32_t to = kCodes ? stage + quarter * L::HALF_CODES
                                     : ring + (base + t) % NS * L::KV_BYTES;
#pragma unroll 4
          for (int i = 0; i < HP; ++i) {
            const long long at = __shfl_sync(0xffffffffu, place, RI * i + sub);
            const bool on = ok && in_row && at >= 0;
            if (!JVP_CHECK(row0 + RI * i + sub < BN, c.status, kChkSmem)) continue;
            if constexpr (kCodes) chunk_copy<8>(to + i * RI * D, rows + (on ? at : 0), on);
            else chunk_copy<16>(to + tile_at(i), rows + (on ? at : 0), on);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      look_up(0);
      resolve();
      look_up(1);
      if (SRC != kChunkStaged) issue(0);
      for (int t = 0; t < n; ++t) {
        const int halves = 4 * (base + t) + quarter, slot = halves % L::AHEAD;
        if constexpr (SRC == kChunkStaged) {
          take(t);
          ok = wait(&ctrl->stage_full[slot], halves / L::AHEAD);
        } else if constexpr (SRC == kChunkRows) {
          issue(t + 1);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        if constexpr (kCodes) {
          ok = ok && wait_empty(t);
          if (!ok) break;
          const uint32_t from = stage + (SRC == kChunkStaged ? slot : quarter) * L::HALF_CODES;
          const uint32_t to = ring + (base + t) % NS * L::KV_BYTES;
          // (a loop: what counts here is the instruction cache, which 20 warps at six
          // different places share.  Unrolled, and with all warps at one half of a tile
          // after the other, a tile of 128 keys at D = 128 took 4.3 us, not 2.25.  Codes
          // moved to T's places by shifts and scaled there by one product, 16-bit, were
          // slower too, 3.0 us: more instructions.)
#pragma unroll 4
          for (int i = 0; i < HP; ++i) {
            uint32_t x[2], y[4];
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(x[0]), "=r"(x[1])
                         : "r"(from + i * RI * D)
                         : "memory");
            const unsigned byte = __shfl_sync(0xffffffffu, scale, RI * i + sub);
            const float f = scale_value(byte);
            e4m3x4_to_half2x2(x[0], y[0], y[1]);
            e4m3x4_to_half2x2(x[1], y[2], y[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = chunk_decode<T>(y[k], f);
            if (JVP_CHECK(row0 + RI * i + sub < BN, c.status, kChkSmem))
              st_shared_v4(to + tile_at(i), y[0], y[1], y[2], y[3]);
          }
          __syncwarp();
          if (SRC == kChunkStaged && lane == 0) mbar_arrive(&ctrl->stage_empty[slot]);
        }
        if (!ok) break;
        if (v && gw == 4 && lane == 0 && g.inspected(t))
          mbar_arrive(&ctrl->v_issued[(seen + g.before(t)) % NS]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[(base + t) % NS]);
        if (SRC == kChunkE4M3) issue(t + 1);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      base += n, seen += g.before(n);
      leave_job(job_k);
    }
  } else {
    // ------------------------------------------------------------ softmax
    if (kGather) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    else if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    if (p.cut && threadIdx.x == THREADS - 1) chunk_name<BN>(p, span);  // (before the first scores)
    __syncwarp();
    const int x = (warp - kSoftmax) >> 2;  // query tile
    const int sub = warp & 3;       // its TMEM lanes 32 sub ..
    const int r = sub * 32 + lane;
    const int rt = r / p.group, rh = r - rt * p.group;  // token and head of the row
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t o_tm = lane_base + L::TM_O + x * D;
    const float scale = p.scale_log2;
    const uint32_t s_tm = lane_base + L::TM_S + x * BN;
    int base = 0, number = 0, uses = 0, stores = 0, steps = 0;
    bool ok = true;
    for (int job_k = 0; ok; ++job_k) {
      const ChunkJob* const job = take_job(job_k);
      if (!job) break;
      const ChunkJob &w = *job, &g = *job;
      ++number;
      const int nx = x ? g.n_b : g.n_a;
      const int first = w.tok0 + x * p.tok;  // first token of the tile
      const int i = first + rt;              // token within the sequence
      const bool row_ok = rt < p.tok && i < w.len;
      // The row sees keys [lo, limit) and the sinks; rows that are not used: all.
      const int at = w.past + i;  // its position
      const int limit = row_ok ? at + 1 : w.keys;
      const int lo = row_ok ? w.see.lo(at) : 0;
      int warp_limit = limit, warp_lo = lo;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        warp_limit = min(warp_limit, __shfl_xor_sync(0xffffffffu, warp_limit, o));
        warp_lo = max(warp_lo, __shfl_xor_sync(0xffffffffu, warp_lo, o));
      }
      float m_run = -INFINITY, l_run = 0.f;  // the base of the exponents, the sum
      for (int t = 0; t < nx; ++t) {
        if (!(ok = wait(&ctrl->s_full[x], steps + t))) break;
        tc_fence_after();
        // The row's visible keys of the tile as bits, where any are hidden: one kind of
        // mask for all reasons, since the loop must stay in the instruction cache.
        const int j0 = g.first_key(t);
        uint32_t missing[4];
        ld_shared_v4(smem_u32(ctrl->missing[(base + t) & 7]), missing);
        const bool masked = j0 + BN > warp_limit || (j0 < warp_lo && j0 + BN > w.see.sinks) ||
                            (missing[0] | missing[1] | missing[2] | missing[3]) != 0u;
        auto visible = [&](int q) {  // keys q .. q + 31
          const int here = limit - (j0 + q);  // keys that are not later than the row's
          uint32_t bits = here >= 32 ? 0xFFFFFFFFu : here <= 0 ? 0u : (1u << here) - 1u;
          const int h0 = max(w.see.sinks - (j0 + q), 0), h1 = min(lo - (j0 + q), 32);
          if (h0 < h1) bits &= ~((0xFFFFFFFFu << h0) & (0xFFFFFFFFu >> (32 - h1)));
          return bits & ~ctrl->missing[(base + t) & 7][q / 32];
        };
        auto hide = [&](float (&y)[32], uint32_t bits) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(bits & (1u << e))) y[e] = -INFINITY;
        };
        // (Gathering leaves the softmax 72 registers fewer: it reads the scores twice,
        // for the maximum and for the weights, in loops that are short for the
        // instruction cache, instead of holding the row.)
        float s[kGather ? 1 : BN], m_tile;
        if constexpr (kGather) {
          m_tile = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < BN; q += 32) {
            uint32_t a[32];
            tmem_ld32(s_tm + q, a);
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(a[e]);
            if (masked) hide(y, visible(q));
            m_tile = fmaxf(m_tile, packed_max(y));
          }
        } else {
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
          if (masked) {
#pragma unroll
            for (int q = 0; q < BN; q += 32) hide(*reinterpret_cast<float(*)[32]>(&s[q]), visible(q));
          }
          m_tile = packed_max(s);
        }
        m_tile *= scale;
        const bool need = m_tile - m_run > PackedElem<T>::kTop;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? packed_base<T>(m_tile) : m_run;
          const float alpha = need ? ex2_approx(m_run - m_new) : 1.f;
          l_run *= alpha;
          m_run = m_new;
          if (t > 0) {
            // (O has tile t - 1's product: these scores were issued behind it)
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
        auto weights = [&](const float (&y)[32], int q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 e2 = fma2(make_float2(y[e], y[e + 1]), c2, nm2);
            e2.x = ex2_approx(e2.x);
            e2.y = ex2_approx(e2.y);
            sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], e2);
            pk[e >> 1] = PackedElem<T>::pack(e2.x, e2.y);
          }
          tmem_st16(s_tm + q / 2, pk);
        };
        if constexpr (kGather) {
#pragma unroll 1
          for (int q = 0; q < BN; q += 32) {
            uint32_t a[32];
            tmem_ld32(s_tm + q, a);
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(a[e]);
            if (masked) hide(y, visible(q));
            weights(y, q);
          }
        } else {
#pragma unroll
          for (int q = 0; q < BN; q += 32) weights(*reinterpret_cast<float(*)[32]>(&s[q]), q);
        }
        l_run += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
                 ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->p_full[x]);
      }
      // ------------------------------------------------------------ epilogue
      if (nx > 0 && ok && (ok = wait(&ctrl->o_full[x], uses))) {
        tc_fence_after();
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (NaN stays NaN)
        const bool in_t = JVP_CHECK(!row_ok || (w.r0 + i < p.T && w.head * p.group + rh < p.H), c.status,
                                    kChkGlobalRow);
        const float lse2 = l_run == 0.f ? -INFINITY
                                        : m_run + PackedElem<T>::kShift +
                                              log2f(l_run * PackedElem<T>::kUnshift);
        const long long ws_row = (static_cast<long long>(w.slot) * NQ + x) * BM + r;
        if (row_ok && in_t) {
          if (w.slot >= 0) p.ws_lse[ws_row] = lse2;
          else if (p.lse)
            p.lse[static_cast<long long>(w.head * p.group + rh) * p.T + w.r0 + i] = lse2 * 0.6931471805599453f;
        }
        // A whole tile of tokens: through the (now idle) Q tile, 16-byte piece k of
        // row r at position k ^ (r % 8), and a TMA store of the box.  Else the
        // sequence ends inside the tile, and each thread writes its row; of a piece,
        // in fp32 to the workspace.
        const bool whole = w.slot < 0 && first + p.tok <= w.len;
        const volatile int* found = ctrl->special[number & 7];
        const int special = (found[0] == number ? 1 : 0) | (found[1] == number ? 2 : 0);
        const uint32_t stage = smem_u32(smem + L::OFF_Q + x * L::Q_BYTES) + r * 128;
        T* dst = static_cast<T*>(p.o) + static_cast<long long>(w.r0 + i) * p.so.n +
                 static_cast<long long>(w.head * p.group + rh) * p.so.h;
        // Sums of the infinities and NaN in columns d .. d + 7 of the values that the
        // row sees among the tiles set apart (weights are positive: infinities keep
        // their sign).
        auto add_special = [&](int d, float (&y)[8]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = 0.f;
          if (d >= c.D) return;
#pragma unroll 1
          for (int t = 0; t < nx; ++t) {
            if (!g.inspected(t) || !(special & (t < g.low ? 1 : 2))) continue;
            const int j1 = min(g.first_key(t) + BN, w.keys);
#pragma unroll 1
            for (int j = g.first_key(t); j < j1; ++j) {
              if (!w.see.sees(at, j)) continue;
              int entry, in_page;
              split_position(c, j, &entry, &in_page);
              const int page = page_of(c, w.b, entry);
              if (page < 0) continue;
              const long long place = page * c.sv.b + w.head * c.sv.h + in_page * c.sv.n + d;
              uint32_t y4[4];
              if constexpr (kCodes) {
                const uint2 codes =
                    __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + place));
                const float f = scale_value(__ldg(
                    c.v_scale + (static_cast<long long>(page) * c.Hkv + w.head) * c.page_size + in_page));
                e4m3x4_to_half2x2(codes.x, y4[0], y4[1]);
                e4m3x4_to_half2x2(codes.y, y4[2], y4[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) y4[k] = chunk_decode<T>(y4[k], f);
              } else {
                const uint4 x4 =
                    __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(c.v) + place));
                y4[0] = x4.x, y4[1] = x4.y, y4[2] = x4.z, y4[3] = x4.w;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t bits = y4[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
                if ((bits & PackedElem<T>::kExp) == PackedElem<T>::kExp) y[k] += PackedElem<T>::get(bits);
              }
            }
          }
        };
#pragma unroll 1
        for (int col = 0; col < D; col += 32) {
          uint32_t o[32];
          tmem_ld32(o_tm + col, o);
          if (special && row_ok) {  // (rare: through local memory, to stay short)
            float sums[32];
#pragma unroll 1
            for (int e = 0; e < 32; e += 8)
              add_special(col + e, *reinterpret_cast<float(*)[8]>(&sums[e]));
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + sums[e]);
          }
          if (w.slot >= 0) {
            if (row_ok && JVP_CHECK(w.slot < 2 * p.grid, c.status, kChkGlobalRow)) {
              float4* to = reinterpret_cast<float4*>(p.ws_o + ws_row * D + col);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                to[e / 4] = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                        __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            }
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t y4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y4[k] = PackedElem<T>::pack(__uint_as_float(o[e + 2 * k]) * inv,
                                         __uint_as_float(o[e + 2 * k + 1]) * inv);
            if (!JVP_CHECK((col / 64) * BM * 128 + r * 128 + 128 <= L::Q_BYTES, c.status, kChkSmem))
              continue;
            if (whole)
              st_shared_v4(stage + (col / 64) * BM * 128 + ((((col % 64 + e) / 8) ^ (r & 7)) << 4),
                           y4[0], y4[1], y4[2], y4[3]);
            else if (row_ok && in_t && col + e < c.D &&
                     JVP_CHECK(col + e + 8 <= c.D, c.status, kChkGlobalCol))
              *reinterpret_cast<uint4*>(dst + col + e) = make_uint4(y4[0], y4[1], y4[2], y4[3]);
          }
        }
        if (whole) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->staged[x]);
          if (warp == kSoftmax + 4 * x && wait(&ctrl->staged[x], stores) && lane == 0) {
            for (int ch = 0; ch < KCH; ++ch)
              tma_store_4d(&maps.o, smem + L::OFF_Q + x * L::Q_BYTES + ch * BM * 128, ch * 64,
                           w.head * p.group, w.r0 + first, 0);
            tma_store_commit();
            tma_store_wait_read();  // shared memory stays valid until then
          }
        }
      }
      if (nx > 0) {
        // (behind this warp's reads of O, and where it stored the tile behind the store's)
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&ctrl->done[x]);
        ++uses;
        if (w.slot < 0 && first + p.tok <= w.len) ++stores;
      }
      steps += nx;
      base += g.n;
      leave_job(job_k);
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
  chunk_tc_kernel<T, D, NQ, SRC>
      <<<static_cast<unsigned>(p.grid), chunk_threads(NQ, SRC), smem, stream>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace jvp
