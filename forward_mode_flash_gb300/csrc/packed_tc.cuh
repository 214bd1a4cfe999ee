// packed_tc.cuh -- attention over packed prompts on the tensor cores
// (tcgen05 + TMEM + TMA), fp16 / bf16, fp32 accumulation.
//
// Per sequence (rows r0 .. r0 + n - 1 of the packed tensors) and query head h:
//   S = scale Q K^T (key j kept for query i if j <= i when causal),
//   O = softmax(S) V, lse = log rowsum(exp S),
// by an online softmax over 128-key tiles.
//
// A query tile is 128 rows of one key/value head: `tok` = 128 / group tokens
// times the `group` query heads that read it (one TMA box {64, group, tok} of
// [T, H, D] lays them out so), so grouped heads share each K/V tile in the same
// product and a short prompt of few tokens still fills rows.  A CTA takes two
// consecutive query tiles A and B of a sequence against the same K/V ring:
// while one tile's softmax runs, the tensor core works for the other.  (NQ = 1,
// for short prompts: one tile, and two CTAs per SM that do the same.)
//   warp 0      TMA producer: Q of both tiles, then K and V tiles through two
//               rings
//   warp 1      TMEM allocator; issues every MMA
//   warp 2      at D = 64 issues MMAs too (below); else only fills the warpgroup
//   warp 3      inspects the V tiles that a mask or the sequence's end cuts
//   warps 4..7  softmax of tile A, one row per thread; warps 8..11 of tile B
//
// The scores of a step (query tile, key tile) are formed in a buffer in TMEM,
// the softmax writes the weights P~ over their first half as 16-bit values, and
// the second product O += P~ V reads them from there as its A operand.  Behind
// the product, in the same warp and therefore in order, go the next scores into
// that buffer: at D = 128 (two buffers; they and both O fill the 512 columns)
// the same tile's, at D = 64 (three) those of three steps on in the order A(0),
// B(0), A(1), B(1), ..., so that a softmax warpgroup finds its next scores
// ready.
//
// The row maximum in the exponent moves only when a tile's maximum exceeds it
// by 2^8 (ratios are exact for any stale maximum), so O is rarely rescaled.
//
// Rounding: the weights are rounded to 16 bits for the second product; the row
// sum adds them unrounded.  bf16 keeps its 8 bits at any size, fp16 its 11 only
// down to 2^-14, where one key far above thousands of others would leave those
// with a few bits, or as zeros.  So fp16 weights are 2^(11 + x - m) and the
// maximum moves past 2^4.9 already (61148 at most, fp16 holds 65504): a weight
// keeps its 11 bits down to 2^-25 of the row's largest (17 nats) and becomes 0
// below 2^-36.  (8192 tokens, 16/16 heads of 64: 295.5 us with the maximum moving
// past 2^8 or 2^5, 297.3 past 2^4, 308.3 past 2^3.)  What is kept is the base
// m - 11 as rounded, and comparisons are of differences from it, so that large
// logits, where fp32 has steps of 1 and more, do not take a weight past its range.
//
// The last key tile of a sequence may end inside the box: the rows behind it
// are another sequence's.  Their scores are replaced before the maximum, and
// their V rows, whose weights are 0, are overwritten with zeros in shared
// memory (0 * NaN would not be 0).  Where a causal mask cuts a tile, its V rows
// are looked through for infinities and NaN while the scores' softmax runs.
// They are rare; if there are any, they too become zeros, and at the end each
// row adds those that it may see.  (The look costs 1 to 2 %, and 0.6 us of 15
// for prompts of one tile.)
//
// What bounds it: at D = 128 the tensor core's operand reads (one step's
// products, 2 x 128 x 128 x 128, read 96 KB of shared memory for 1024 cycles of
// tensor work at 128 bytes a cycle, and copies write 32 KB more); at D = 64 the
// exponentials and the rest of the softmax; prompts of a few tiles, a CTA's
// beginning and end (about 3 us of set-up, first loads and stores).  Measured,
// bf16, 16/2 heads of 128, causal, 16384 and 10101 tokens: 914 us in short runs,
// 1660 TFLOP/s (tensor pipe 70 % active), 980 us after a second, under the power
// cap; fp16, 16/16 heads of 64, 8192 tokens: 293 us, 938 TFLOP/s; bf16, 16/4
// heads of 128, causal, twelve of 166 to 2048 tokens: 88 us, 896 TFLOP/s.
// Measured and not kept: a persistent CTA that takes over blocks
// through the launch control (8 % slower on long prompts: its item rings keep
// more warps polling; 20 % faster on prompts of one tile); at D = 128, one
// issuing warp per query tile (the tiles' products interleave and both scores
// come late: 1182 against 1154 us); waits with a suspend-time hint (5 % slower).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "debug_checks.cuh"
#include "packed.cuh"
#include "sm103_ptx.cuh"

namespace jvp {

template <typename T>
struct PackedElem;
template <>
struct PackedElem<__half> {
  static constexpr bool kBF16 = false;
  // weights are 2^(x - base), the base kShift below a maximum; it moves where they
  // would pass 2^kTop
  static constexpr float kShift = 11.f, kUnshift = 1.f / 2048.f, kTop = 15.9f;
  static constexpr uint32_t kExp = 0x7C00u;  // exponent bits, all set: infinity or NaN
  static __device__ __forceinline__ float get(uint32_t bits) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // acc + 0 x: not zero once an x was an infinity or NaN
  static __device__ __forceinline__ void zeros(uint32_t x, uint32_t* acc) {
    __half2* a = reinterpret_cast<__half2*>(acc);
    *a = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.f), *a);
  }
};
template <>
struct PackedElem<__nv_bfloat16> {
  static constexpr bool kBF16 = true;
  static constexpr float kShift = 0.f, kUnshift = 1.f, kTop = 8.f;
  static constexpr uint32_t kExp = 0x7F80u;
  static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void zeros(uint32_t x, uint32_t* acc) {
    __nv_bfloat162* a = reinterpret_cast<__nv_bfloat162*>(acc);
    *a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), __float2bfloat162_rn(0.f), *a);
  }
};

template <int D, int NQ>
struct PackedLayout {
  static constexpr int BM = kPackedTileRows, BN = kPackedBlockN;
  static constexpr int KCH = D / 64;             // 128-byte chunks along D
  // stages of each ring
  static constexpr int NS = NQ == 2 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 2);
  static constexpr int Q_BYTES = KCH * BM * 128; // one query tile
  static constexpr int KV_BYTES = KCH * BN * 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQ * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NS * KV_BYTES;
  static constexpr int OFF_CTRL = OFF_V + NS * KV_BYTES;
  static constexpr int SMEM_BYTES = OFF_CTRL + 1024 + 1024;  // control block, alignment
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert((3 - NQ) * (SMEM_BYTES + 1024) <= 228 * 1024 &&
                    (4 - NQ) * (SMEM_BYTES + 1024) > 228 * 1024,
                "3 - NQ CTAs per SM, which share the TMEM columns");
  static constexpr int NB = NQ == 1 ? 1 : D == 128 ? 2 : 3;  // score buffers
  static constexpr uint32_t TM_S = 0;            // S / P~ of buffer b at b * BN
  static constexpr uint32_t TM_O = NB * BN;      // O of tile x at TM_O + x * D
  static constexpr uint32_t TM_COLS = NQ * 256;
  static_assert(NB * BN + NQ * D <= TM_COLS, "TMEM columns");
};

// One warpgroup for the copies and the MMAs and one for the softmax of each
// query tile.  A softmax thread holds a whole row of scores, so its group
// takes registers from the first (of 384 threads: 168 * 3 = 72 + 2 * 216; of
// 256: 128 * 2 = 48 + 208).
constexpr int packed_threads(int NQ) { return 128 + 128 * NQ; }

template <int NS>
struct PackedCtrl {
  uint64_t q_full[2];
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  // By inspected V tile modulo NS: its copy has begun (so that its v_full phase
  // is the barrier's current one or over); it may be used.
  uint64_t v_issued[NS], v_checked[NS];
  // By query tile and, with three buffers, by key tile modulo 3.  (A parity
  // cannot tell a phase from the one two before or behind it, so a waiter must
  // know the phase before to be over and the one behind not to be.  With three
  // buffers the two issuing warps drive each other, and a tile's scores and
  // weights can be up to three key tiles ahead of its own products.)
  uint64_t s_full[2][3];  // scores against the next key tile are final
  uint64_t p_full[2][3];  // its P~ is stored
  uint64_t o_done[2][3];  // O has its product (NB = 3)
  uint64_t o_full[2];     // O has the last key tile's product
  uint64_t staged[2];   // the tile's output rows are in shared memory
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  int special;  // V entries were infinite or NaN where the mask cuts a tile
};

__device__ __forceinline__ void packed_timeout(unsigned int* status, volatile int* abort) {
  *abort = 1;
  atomicOr(status, 1u);
}
// Bounded wait by every lane, with a warp-uniform outcome (the TMEM
// instructions that follow are warp-collective).
__device__ __forceinline__ bool packed_warp_wait(uint64_t* bar, uint32_t parity,
                                                 unsigned int* status, volatile int* abort) {
  const bool got = mbar_wait<false>(bar, parity, abort);
  if (!got) packed_timeout(status, abort);
  return __all_sync(0xffffffffu, got);
}

// Maximum of 2^k values by three-input maxima.
template <int N>
__device__ __forceinline__ float packed_max(const float (&x)[N]) {
  float y[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i + 8 <= N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = fmax3(y[k], x[i + k], x[i + 4 + k]);
  y[0] = fmax3(y[0], x[N - 4], x[N - 3]);
  y[1] = fmax3(y[1], x[N - 2], x[N - 1]);
  return fmaxf(fmax3(y[0], y[1], y[2]), y[3]);
}

// Base of the exponents for a maximum m (m itself where a step of fp32 is 16, so
// that m - 11 would be m - 16).
template <typename T>
__device__ __forceinline__ float packed_base(float m) {
  const float b = m - PackedElem<T>::kShift;
  return m - b > PackedElem<T>::kTop ? m : b;
}

template <typename T, int D, int NQ>
__global__ void __launch_bounds__(packed_threads(NQ), 3 - NQ)
    packed_tc_kernel(const __grid_constant__ PackedMaps maps, const PackedParams p) {
  using L = PackedLayout<D, NQ>;
  constexpr int BM = L::BM, BN = L::BN, NS = L::NS, NB = L::NB, KCH = L::KCH;
  constexpr bool kBF16 = PackedElem<T>::kBF16;
  constexpr uint32_t IDESC_S = idesc_f16(kBF16, BM, BN, false);
  constexpr uint32_t IDESC_O = idesc_f16(kBF16, BM, D, true);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using Ctrl = PackedCtrl<NS>;
  static_assert(sizeof(Ctrl) <= 1024, "control block budget");
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + L::OFF_CTRL);
  volatile int* abort = &ctrl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Set-up first, so that it runs while the offsets are fetched.
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
      mbar_init(&ctrl->k_full[s], 1);
      mbar_init(&ctrl->k_empty[s], NB == 3 ? 2 : 1);  // one arrival per issuing warp
      mbar_init(&ctrl->v_full[s], 1);
      mbar_init(&ctrl->v_empty[s], NB == 3 ? 2 : 1);
      mbar_init(&ctrl->v_issued[s], 1);
      mbar_init(&ctrl->v_checked[s], 1);
    }
    ctrl->abort = 0;
    ctrl->special = 0;
    fence_barrier_init();
  }
  __syncwarp();
  // Key/value heads in groups whose rows stay in L2, the heads of a group
  // innermost; causal sequences begin with their last (longest) tile.
  const int per_group = p.tiles * p.head_group;
  const int hg = static_cast<int>(blockIdx.x) / per_group;
  const int in_group = static_cast<int>(blockIdx.x) - hg * per_group;
  const int heads = min(p.head_group, p.Hkv - hg * p.head_group);
  const int hk = hg * p.head_group + in_group % heads;
  const int u = in_group / heads;
  PackedTile pt;
  const bool have = find_packed_tile(p.cu, p.B, p.T, NQ * p.tok, u, p.causal != 0, p.status, &pt);
  if (!have) return;  // (the list is shorter than its bound; the same for every warp)
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, L::TM_COLS);
    tmem_relinquish();
  }
  const int len = pt.len, r0 = pt.r0;
  const int tok0 = pt.tile * NQ * p.tok;  // first token of tile A; B follows
  // key tiles of a query tile whose first token is a
  auto key_tiles = [&](int a) {
    if (a >= len) return 0;
    const int keys = p.causal ? min(a + p.tok, len) : len;
    return (keys + BN - 1) / BN;
  };
  const int n_a = key_tiles(tok0), n_b = NQ == 2 ? key_tiles(tok0 + p.tok) : 0;
  const int n = max(n_a, n_b), both = min(n_a, n_b);
  // V tiles from this one on are inspected: a mask hides some of their keys
  // from some rows, or the sequence ends inside
  const int inspect = p.causal ? tok0 / BN : len % BN ? n - 1 : n;
  // score buffer of query tile x against key tile t: steps go A(0), B(0), A(1),
  // ... round the three buffers; of two, each tile has its own
  auto buffer_of = [&](int x, int t) {
    return NB <= 2 ? x : (t < both ? 2 * t + x : both + t) % NB;
  };
  // which of a tile's barriers is key tile t's, and its phase
  auto bar_of = [&](int t) { return NB == 3 ? t % 3 : 0; };
  auto phase_of = [&](int t) { return NB == 3 ? t / 3 : t; };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return packed_warp_wait(bar, parity & 1, p.status, abort);
  };

  if (warp < 4) {
    if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      bool ok = true;
      if (lane == 0) {
        auto load_q = [&](int x) {
          mbar_arrive_expect_tx(&ctrl->q_full[x], KCH * p.group * p.tok * 128);
          for (int c = 0; c < KCH; ++c)
            tma_load_4d(smem + L::OFF_Q + x * L::Q_BYTES + c * BM * 128, &maps.q, &ctrl->q_full[x],
                        c * 64, hk * p.group, r0 + tok0 + x * p.tok, 0);
        };
        int k_fills = 0, v_fills = 0;
        auto load_kv = [&](int t, bool v) -> bool {
          const int s = t % NS;
          uint64_t* empty = v ? &ctrl->v_empty[s] : &ctrl->k_empty[s];
          uint64_t* full = v ? &ctrl->v_full[s] : &ctrl->k_full[s];
          if (!mbar_wait<false>(empty, ((t / NS) & 1) ^ 1, abort)) return false;
          mbar_arrive_expect_tx(full, L::KV_BYTES);
          uint8_t* dst = smem + (v ? L::OFF_V : L::OFF_K) + s * L::KV_BYTES;
          for (int c = 0; c < KCH; ++c)
            tma_load_4d(dst + c * BN * 128, v ? &maps.v : &maps.k, full, c * 64, r0 + t * BN, hk,
                        0);
          if (v && t >= inspect) mbar_arrive(&ctrl->v_issued[(t - inspect) % NS]);
          ++(v ? v_fills : k_fills);
          return true;
        };
        load_q(0);
        ok = load_kv(0, false);
        if (n_b > 0) load_q(1);
        for (int t = 0; ok && t < n; ++t) {
          ok = load_kv(t, true);
          if (ok && t + 1 < n) ok = load_kv(t + 1, false);
        }
        if (!ok) {
          packed_timeout(p.status, abort);
          // let every copy already issued land before the CTA can exit
          const int zero = 0;
          mbar_wait(&ctrl->q_full[0], 0, &zero);
          if (n_b > 0) mbar_wait(&ctrl->q_full[1], 0, &zero);
          for (int t = max(0, k_fills - NS); t < k_fills; ++t)
            mbar_wait(&ctrl->k_full[t % NS], (t / NS) & 1, &zero);
          for (int t = max(0, v_fills - NS); t < v_fills; ++t)
            mbar_wait(&ctrl->v_full[t % NS], (t / NS) & 1, &zero);
        }
      }
    } else if (warp == 1 || (NB == 3 && warp == 2)) {
      // ---------------------------------------------------------- MMAs
      // The whole warp walks the steps; one elected lane issues.  (Descriptor
      // addresses are in units of 16 bytes.)
      const int w = warp - 1;
      const uint32_t neg_a = p.neg_scores ? (1u << 13) : 0u;
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::OFF_V), BN * 128, 1024);
      // The pace of this warp is the kernel's: between two products there is
      // little but their waits, and the buffers of the main loops are constants.
      auto scores = [&](int x, int t, int buf, int bar) {
        const uint64_t qd = q_desc + x * (L::Q_BYTES >> 4);
        const uint64_t kd = k_desc + (t % NS) * (L::KV_BYTES >> 4);
#pragma unroll
        for (int c = 0; c < KCH; ++c)
          mma_ss_x4_warp<2, 2>(tmem + L::TM_S + buf * BN, qd + c * (BM * 128 / 16),
                               kd + c * (BN * 128 / 16), IDESC_S | neg_a, c > 0 ? 1u : 0u);
        mma_commit_warp(&ctrl->s_full[x][bar]);
      };
      auto k_landed = [&](int t) {
        const bool got = wait(&ctrl->k_full[t % NS], t / NS);
        tc_fence_after();
        return got;
      };
      auto v_landed = [&](int t) {
        const int k = t - inspect;
        return k < 0 ? wait(&ctrl->v_full[t % NS], t / NS) : wait(&ctrl->v_checked[k % NS], k / NS);
      };
      // O of query tile x: the product with the weights in buffer buf.  (The
      // tensor core runs one warp's products in order: scores issued behind it
      // may overwrite the weights.)
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
        // Two issuing warps, each releasing every K and V tile once.  While
        // both query tiles have keys, warp w has tile w's products; behind
        // step i's come the scores of step i + 3 (the other tile's) into the
        // same buffer: tile A's product is followed by B's scores one key tile
        // on, B's by A's two key tiles on.
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
        // Then one tile alone, issued by its own warp, its scores two key tiles
        // ahead of its products.  (B goes on alone for at most one key tile, as
        // its tokens end at most 128 behind A's: that step's buffer is the one
        // that B's own product against tile both - 2 has released.)
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
      if (!ok) packed_timeout(p.status, abort);
      // every MMA issued completes before TMEM is freed
      mma_commit_warp(&ctrl->drain[w]);
      const int zero = 0;
      mbar_wait(&ctrl->drain[w], 0, &zero);
    } else if (warp == 3) {
      // ---------------------------------------------------------- V inspector
      // (A tile's copy may begin only when the products of the tile NS before
      // are done, so one barrier per stage will do, as for the copies.)
      bool ok = true;
      for (int t = inspect; ok && t < n; ++t) {
        const int k = t - inspect;
        ok = wait(&ctrl->v_issued[k % NS], k / NS) && wait(&ctrl->v_full[t % NS], t / NS);
        if (!ok) break;
        const uint32_t v = smem_u32(smem + L::OFF_V + t % NS * L::KV_BYTES);
        const int rows = min(BN, len - t * BN);
        const int from = max(0, tok0 + 1 - t * BN);  // rows before: every token sees them
        for (int e = lane; e < (BN - rows) * KCH * 8; e += 32) {
          const int piece = e % 8, c = (e / 8) % KCH, row = rows + e / (8 * KCH);
          if (JVP_CHECK(row < BN, p.status, kChkSmem))
            st_shared_v4(v + c * BN * 128 + row * 128 + piece * 16, 0u, 0u, 0u, 0u);
        }
        if (p.causal && from < rows) {
          using E = PackedElem<T>;
          uint32_t seen[4] = {0u, 0u, 0u, 0u};
          for (int c = 0; c < KCH; ++c) {
            const uint32_t base = v + c * BN * 128;
#pragma unroll 4
            for (int e = from * 8 + lane; e < rows * 8; e += 32) {
              uint32_t x[4];
              ld_shared_v4(base + e * 16, x);
#pragma unroll
              for (int i = 0; i < 4; ++i) E::zeros(x[i], &seen[i]);
            }
          }
          const uint32_t any = seen[0] | seen[1] | seen[2] | seen[3];
          if (__any_sync(0xffffffffu, (any & 0x7FFF7FFFu) != 0u)) {
            for (int c = 0; c < KCH; ++c)
              for (int e = from * 8 + lane; e < rows * 8; e += 32) {
                uint32_t x[4];
                if (!JVP_CHECK(e * 16 + 16 <= BN * 128, p.status, kChkSmem)) continue;
                ld_shared_v4(v + c * BN * 128 + e * 16, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((x[i] & E::kExp) == E::kExp) x[i] &= 0xFFFF0000u;
                  if ((x[i] >> 16 & E::kExp) == E::kExp) x[i] &= 0x0000FFFFu;
                }
                st_shared_v4(v + c * BN * 128 + e * 16, x[0], x[1], x[2], x[3]);
              }
            if (lane == 0) *static_cast<volatile int*>(&ctrl->special) = 1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->v_checked[k % NS]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - 4) >> 2;  // query tile
    const int sub = warp & 3;       // its TMEM lanes 32 sub ..
    const int r = sub * 32 + lane;
    const int nx = x ? n_b : n_a;
    const int rt = r / p.group, rh = r - rt * p.group;  // token and head of the row
    const int first = tok0 + x * p.tok;                 // first token of the tile
    const int i = first + rt;                           // token within the sequence
    const bool row_ok = rt < p.tok && i < len;
    // keys j < limit count; for the rows of the tile that are not used: all
    const int limit = (p.causal && row_ok) ? i + 1 : len;
    int warp_limit = limit;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      warp_limit = min(warp_limit, __shfl_xor_sync(0xffffffffu, warp_limit, o));
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t o_tm = lane_base + L::TM_O + x * D;
    const float c = p.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;  // the base of the exponents, the sum
    bool ok = true;
    for (int t = 0; t < nx; ++t) {
      const uint32_t s_tm = lane_base + L::TM_S + buffer_of(x, t) * BN;
      if (!(ok = wait(&ctrl->s_full[x][bar_of(t)], phase_of(t)))) break;
      tc_fence_after();
      float s[BN];
      const bool s_cols = JVP_CHECK(buffer_of(x, t) < NB && buffer_of(x, t) >= 0, p.status, kChkTmem);
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
      const int j0 = t * BN;
      if (j0 + BN > warp_limit) {
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (j0 + e >= limit) s[e] = -INFINITY;
      }
      const float m_tile = packed_max(s) * c;
      const bool need = m_tile - m_run > PackedElem<T>::kTop;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? packed_base<T>(m_tile) : m_run;
        const float alpha = need ? ex2_approx(m_run - m_new) : 1.f;
        l_run *= alpha;
        m_run = m_new;
        if (t > 0) {
          // O has tile t - 1's product: with up to two buffers because these
          // scores were issued behind it, with three by the barrier.  (Its
          // phase before, tile t - 4's product, is over: these scores were
          // issued behind the other tile's product of t - 2 or t - 1, whose
          // weights come from scores that were committed behind this tile's
          // product of t - 3; alone, behind its own of t - 2.)
          if (NB == 3) {
            if (!(ok = wait(&ctrl->o_done[x][bar_of(t - 1)], phase_of(t - 1)))) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            if (!JVP_CHECK(L::TM_O + x * D + col + 32 <= L::TM_COLS, p.status, kChkTmem)) continue;
            uint32_t o[32];
            tmem_ld32(o_tm + col, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_tm + col, o);
          }
        }
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      const float2 c2 = make_float2(c, c), nm2 = make_float2(-m_use, -m_use);
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
      const bool in_t = JVP_CHECK(!row_ok || (r0 + i < p.T && hk * p.group + rh < p.H), p.status,
                                  kChkGlobalRow);
      if (row_ok && p.lse && in_t)
        p.lse[static_cast<long long>(hk * p.group + rh) * p.T + r0 + i] =
            l_run == 0.f ? -INFINITY
                         : (m_run + PackedElem<T>::kShift + log2f(l_run * PackedElem<T>::kUnshift)) *
                               0.6931471805599453f;
      // All tokens of the tile exist: through the (now idle) Q tile, 16-byte
      // piece k of row r at position k ^ (r % 8), and a TMA store of the box.
      // Else the sequence ends inside the tile: each thread writes its row.
      const bool whole = first + p.tok <= len;
      const bool special = *static_cast<volatile int*>(&ctrl->special) != 0;
      const uint32_t stage = smem_u32(smem + L::OFF_Q + x * L::Q_BYTES) + r * 128;
      T* dst = static_cast<T*>(p.o) + static_cast<long long>(r0 + i) * p.so.n +
               static_cast<long long>(hk * p.group + rh) * p.so.h;
#pragma unroll
      for (int col = 0; col < D; col += 64) {
        uint32_t o[2][32];
        tmem_ld32x2(o_tm + col, o_tm + col + 32, o[0], o[1]);
        if (special && row_ok) {  // weights are positive: infinities keep their sign
          const T* vs = static_cast<const T*>(p.v) + static_cast<long long>(r0) * p.sv.n +
                        static_cast<long long>(hk) * p.sv.h + col;
#pragma unroll 1
          for (int j = tok0 + 1; j <= i; ++j)
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
              uint4 y = make_uint4(0u, 0u, 0u, 0u);
              if (col + e < p.D)
                y = __ldg(reinterpret_cast<const uint4*>(vs + static_cast<long long>(j) * p.sv.n + e));
              const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t bits = w[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
                if ((bits & PackedElem<T>::kExp) == PackedElem<T>::kExp) {
                  uint32_t& to = o[(e + k) / 32][(e + k) % 32];
                  to = __float_as_uint(__uint_as_float(to) + PackedElem<T>::get(bits));
                }
              }
            }
        }
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = PackedElem<T>::pack(__uint_as_float(o[e / 32][e % 32 + 2 * k]) * inv,
                                       __uint_as_float(o[e / 32][e % 32 + 2 * k + 1]) * inv);
          if (!JVP_CHECK((col / 64) * BM * 128 + r * 128 + 128 <= L::Q_BYTES, p.status, kChkSmem))
            continue;
          if (whole)
            st_shared_v4(stage + (col / 64) * BM * 128 + (((e / 8) ^ (r & 7)) << 4), w[0], w[1],
                         w[2], w[3]);
          else if (row_ok && in_t && col + e < p.D &&
                   JVP_CHECK(col + e + 8 <= p.D, p.status, kChkGlobalCol))
            *reinterpret_cast<uint4*>(dst + col + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (whole) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->staged[x]);
        if (warp == 4 + 4 * x && wait(&ctrl->staged[x], 0) && lane == 0) {
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

template <typename T, int D, int NQ>
cudaError_t launch_packed_tc_variant(const PackedMaps& maps, const PackedParams& p,
                                     cudaStream_t stream) {
  constexpr int smem = PackedLayout<D, NQ>::SMEM_BYTES;
  const cudaError_t e = allow_shared_memory<packed_tc_kernel<T, D, NQ>>(smem);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.tiles) * p.Hkv;
  packed_tc_kernel<T, D, NQ>
      <<<static_cast<unsigned>(grid), packed_threads(NQ), smem, stream>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace jvp
