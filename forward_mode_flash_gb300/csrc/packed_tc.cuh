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
// while one tile's softmax runs, the tensor core works for the other.
//   warp 0      TMA producer: Q of both tiles, then K and V tiles through two
//               rings
//   warp 1      TMEM allocator; issues every MMA:
//               S_A(t + 1) right after O_A += P_A(t) V(t), then the same for B
//   warps 4..7  softmax of tile A, one row per thread; warps 8..11 of tile B
// P~ overwrites the first half of its S columns as 16-bit values and is the A
// operand of the second product from TMEM; it is published in two halves, so
// that the product starts while the second half's exponentials are formed.  MMAs of one thread complete in
// order, so "S(t + 1) is final" also says that O has tile t's contribution:
// the (rare) rescale of O needs no barrier of its own.
//
// The row maximum in the exponent moves only when a tile's maximum exceeds it
// by 2^8; ratios are exact for any stale maximum.
//
// The last key tile of a sequence may end inside the box: the rows behind it
// are another sequence's.  Their scores are replaced before the maximum, and
// their V rows, whose weights are 0, are overwritten with zeros in shared
// memory (0 * NaN would not be 0).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "debug_checks.cuh"
#include "packed.cuh"
#include "sm103_ptx.cuh"

namespace jvp {

template <typename T>
struct PackedElem;
template <>
struct PackedElem<__half> {
  static constexpr bool kBF16 = false;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct PackedElem<__nv_bfloat16> {
  static constexpr bool kBF16 = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <int D>
struct PackedLayout {
  static constexpr int BM = kPackedTileRows, BN = kPackedBlockN;
  static constexpr int KCH = D / 64;             // 128-byte chunks along D
  static constexpr int NS = D == 128 ? 2 : 4;    // stages of each ring
  static constexpr int Q_BYTES = KCH * BM * 128; // one query tile
  static constexpr int KV_BYTES = KCH * BN * 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NS * KV_BYTES;
  static constexpr int OFF_CTRL = OFF_V + NS * KV_BYTES;
  static constexpr int SMEM_BYTES = OFF_CTRL + 1024 + 1024;  // control block, alignment
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(SMEM_BYTES > 114 * 1024, "one CTA per SM: it owns all TMEM columns");
  static constexpr uint32_t TM_S = 0;            // S / P~ of tile x at x * BN
  static constexpr uint32_t TM_O = 2 * BN;       // O of tile x at TM_O + x * D
  static constexpr uint32_t TM_COLS = 512;
};

// Three warpgroups: producer and MMA warps (two more only fill the group),
// softmax of tile A, softmax of tile B.  A softmax thread holds a whole row of
// scores, so its group takes registers from the first (168 * 3 = 72 + 2 * 216).
constexpr int kPackedThreads = 384;

template <int NS>
struct PackedCtrl {
  uint64_t q_full[2];
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t v_tail;     // the last V tile's rows behind the sequence are zero
  uint64_t s_full[2];  // S of the next key tile is final (and O has the previous one's)
  uint64_t p_half[2];  // P~ of the tile's first 64 keys is stored
  uint64_t p_full[2];  // P~ of the others is
  uint64_t o_full[2];  // O is complete
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void packed_timeout(unsigned int* status, volatile int* abort) {
  *abort = 1;
  atomicOr(status, 1u);
}
// Bounded wait by every lane, with a warp-uniform outcome (the TMEM
// instructions that follow are warp-collective).
__device__ __forceinline__ bool packed_warp_wait(uint64_t* bar, uint32_t parity,
                                                 unsigned int* status, volatile int* abort) {
  const bool got = mbar_wait(bar, parity, abort);
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

template <typename T, int D>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_tc_kernel(const __grid_constant__ PackedMaps maps, const PackedParams p) {
  using L = PackedLayout<D>;
  constexpr int BM = L::BM, BN = L::BN, NS = L::NS, KCH = L::KCH;
  constexpr bool kBF16 = PackedElem<T>::kBF16;
  constexpr uint32_t IDESC_S = idesc_f16(kBF16, BM, BN, false);
  constexpr uint32_t IDESC_O = idesc_f16(kBF16, BM, D, true);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  static_assert(sizeof(PackedCtrl<NS>) <= 1024, "control block budget");
  PackedCtrl<NS>* ctrl = reinterpret_cast<PackedCtrl<NS>*>(smem + L::OFF_CTRL);
  volatile int* abort = &ctrl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Heads outermost, so that the CTAs in flight share a key/value head's rows
  // in L2; causal sequences begin with their last (longest) tile.
  const int hk = static_cast<int>(blockIdx.x) / p.tiles;
  const int u = static_cast<int>(blockIdx.x) % p.tiles;
  PackedTile pt;
  if (!find_packed_tile(p.cu, p.B, p.T, 2 * p.tok, u, p.causal != 0, p.status, &pt)) return;
  const int len = pt.len, r0 = pt.r0;
  const int tok0 = pt.tile * 2 * p.tok;  // first token of tile A; B follows
  // key tiles of a query tile whose first token is a
  auto key_tiles = [&](int a) {
    if (a >= len) return 0;
    const int keys = p.causal ? min(a + p.tok, len) : len;
    return (keys + BN - 1) / BN;
  };
  const int n_a = key_tiles(tok0), n_b = key_tiles(tok0 + p.tok);
  const int n = max(n_a, n_b);
  const int tail = len - (n - 1) * BN;  // keys of the last tile (>= BN: all of its rows)

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctrl->q_full[x], 1);
      mbar_init(&ctrl->s_full[x], 1);
      mbar_init(&ctrl->p_half[x], 4);  // one arrival per softmax warp of the tile
      mbar_init(&ctrl->p_full[x], 4);
      mbar_init(&ctrl->o_full[x], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&ctrl->k_full[s], 1);
      mbar_init(&ctrl->k_empty[s], 1);
      mbar_init(&ctrl->v_full[s], 1);
      mbar_init(&ctrl->v_empty[s], 1);
    }
    mbar_init(&ctrl->v_tail, 1);
    mbar_init(&ctrl->drain, 1);
    ctrl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, L::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    if (lane == 0) {
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
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
        if (!mbar_wait(empty, ((t / NS) & 1) ^ 1, abort)) return false;
        mbar_arrive_expect_tx(full, L::KV_BYTES);
        uint8_t* dst = smem + (v ? L::OFF_V : L::OFF_K) + s * L::KV_BYTES;
        for (int c = 0; c < KCH; ++c)
          tma_load_4d(dst + c * BN * 128, v ? &maps.v : &maps.k, full, c * 64, r0 + t * BN, hk, 0);
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
    ok = __all_sync(0xffffffffu, ok);
    if (ok && tail < BN) {
      // rows of the last V tile behind the sequence: zero
      const int t = n - 1, s = t % NS;
      ok = packed_warp_wait(&ctrl->v_full[s], (t / NS) & 1, p.status, abort);
      if (ok) {
        const uint32_t v = smem_u32(smem + L::OFF_V + s * L::KV_BYTES);
        for (int e = lane; e < (BN - tail) * KCH * 8; e += 32) {
          const int piece = e % 8, c = (e / 8) % KCH, row = tail + e / (8 * KCH);
          st_shared_v4(v + c * BN * 128 + row * 128 + piece * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->v_tail);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    // The whole warp walks this loop; one elected lane issues.
    const uint32_t neg_a = p.neg_scores ? (1u << 13) : 0u;
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::OFF_V), BN * 128, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool got = packed_warp_wait(bar, parity, p.status, abort);
      tc_fence_after();
      return got;
    };
    // S of tile x against key tile t (whose K has landed).  (Descriptor
    // addresses are in units of 16 bytes.)
    auto scores = [&](int x, int t) {
      const uint64_t q = q_desc + x * (L::Q_BYTES >> 4);
      const uint64_t k = k_desc + (t % NS) * (L::KV_BYTES >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_warp(tmem + L::TM_S + x * BN, q + ((kk >> 2) * BM * 128 + (kk & 3) * 32) / 16,
                    k + ((kk >> 2) * BN * 128 + (kk & 3) * 32) / 16, IDESC_S | neg_a,
                    kk > 0 ? 1u : 0u);
      mma_commit_warp(&ctrl->s_full[x]);
    };
    // O of tile x: the products of half a key tile
    auto values = [&](int x, int t, int half) {
      const uint64_t v = v_desc + (t % NS) * (L::KV_BYTES >> 4);
#pragma unroll
      for (int k2 = 0; k2 < BN / 32; ++k2) {
        const int kk = half * (BN / 32) + k2;
        mma_ts_warp(tmem + L::TM_O + x * D, tmem + L::TM_S + x * BN + kk * 8,
                    v + kk * (16 * 128 / 16), IDESC_O, (t > 0 || kk > 0) ? 1u : 0u);
      }
    };
    bool ok = wait(&ctrl->q_full[0], 0) && wait(&ctrl->k_full[0], 0);
    if (ok) {
      scores(0, 0);
      if (n_b > 0) {
        ok = wait(&ctrl->q_full[1], 0);
        if (ok) scores(1, 0);
      }
      mma_commit_warp(&ctrl->k_empty[0]);
    }
    for (int t = 0; ok && t < n; ++t) {
      const bool b_last = t < n_b;           // B is the last user of V(t) ...
      const bool b_last_k = t + 1 < n_b;     // ... and of K(t + 1)
      bool v_here = false, k_here = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int nx = x ? n_b : n_a;
        if (!ok || t >= nx) continue;
        if (!v_here)
          ok = (t == n - 1 && tail < BN) ? wait(&ctrl->v_tail, 0)
                                         : wait(&ctrl->v_full[t % NS], (t / NS) & 1);
        v_here = true;
        if (!ok || !(ok = wait(&ctrl->p_half[x], t & 1))) continue;
        values(x, t, 0);
        if (!(ok = wait(&ctrl->p_full[x], t & 1))) continue;
        values(x, t, 1);
        if (b_last ? x == 1 : x == 0) mma_commit_warp(&ctrl->v_empty[t % NS]);
        if (t + 1 < nx) {
          if (!k_here && !(ok = wait(&ctrl->k_full[(t + 1) % NS], ((t + 1) / NS) & 1))) continue;
          k_here = true;
          scores(x, t + 1);
          if (b_last_k ? x == 1 : x == 0) mma_commit_warp(&ctrl->k_empty[(t + 1) % NS]);
        } else {
          mma_commit_warp(&ctrl->o_full[x]);
        }
      }
    }
    // every MMA issued completes before TMEM is freed
    mma_commit_warp(&ctrl->drain);
    const int zero = 0;
    mbar_wait(&ctrl->drain, 0, &zero);
  }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int x = (warp - 4) >> 2;  // query tile
    const int sub = warp & 3;       // its TMEM lanes 32 sub ..
    const int r = sub * 32 + lane;
    const int nx = x ? n_b : n_a;
    const int i = tok0 + x * p.tok + r / p.group;  // token within the sequence
    const int h = hk * p.group + r % p.group;
    const bool row_ok = r < p.tok * p.group && i < len;
    // keys j < limit count; for the rows of the tile that are not used: all
    const int limit = (p.causal && row_ok) ? i + 1 : len;
    int warp_limit = limit;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      warp_limit = min(warp_limit, __shfl_xor_sync(0xffffffffu, warp_limit, o));
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t s_tm = lane_base + L::TM_S + x * BN, o_tm = lane_base + L::TM_O + x * D;
    const float c = p.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int t = 0; t < nx; ++t) {
      if (!packed_warp_wait(&ctrl->s_full[x], t & 1, p.status, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[BN];
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
      const bool need = m_tile > m_run + 8.f;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? m_tile : m_run;
        const float alpha = need ? ex2_approx(m_run - m_new) : 1.f;
        l_run *= alpha;
        m_run = m_new;
        if (t > 0) {
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
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
        if (q == BN / 2 - 32) {  // the second product starts on the first half
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->p_half[x]);
        }
      }
      l_run += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
               ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->p_full[x]);
    }
    // ------------------------------------------------------------ epilogue
    if (nx > 0 && ok) ok = packed_warp_wait(&ctrl->o_full[x], 0, p.status, abort);
    if (nx > 0 && ok) {
      tc_fence_after();
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (NaN stays NaN)
      if (row_ok && p.lse)
        p.lse[static_cast<long long>(h) * p.T + r0 + i] =
            l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
      // Rows through the (now idle) Q tile, so that a warp's stores cover
      // whole rows; 16-byte piece k of row r at position k ^ (r % 8).
      constexpr int PIECES = D / 8;
      const uint32_t stage = smem_u32(smem + L::OFF_Q + x * L::Q_BYTES);
#pragma unroll
      for (int col = 0; col < D; col += 32) {
        uint32_t o[32];
        tmem_ld32(o_tm + col, o);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = PackedElem<T>::pack(__uint_as_float(o[e + 2 * k]) * inv,
                                       __uint_as_float(o[e + 2 * k + 1]) * inv);
          const int piece = (col + e) / 8;
          st_shared_v4(stage + r * (D * 2) + ((piece ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      const int piece = lane % PIECES, d = piece * 8;
#pragma unroll 4
      for (int k = 0; k < 32; k += 32 / PIECES) {
        const int rr = sub * 32 + k + lane / PIECES;
        const int ii = tok0 + x * p.tok + rr / p.group;
        const float4 w = ld_shared_v4f(stage + rr * (D * 2) + ((piece ^ (rr & 7)) << 4));
        if (rr < p.tok * p.group && ii < len && d < p.D) {
          T* dst = static_cast<T*>(p.o) + static_cast<long long>(r0 + ii) * p.so.n +
                   static_cast<long long>(hk * p.group + rr % p.group) * p.so.h + d;
          *reinterpret_cast<float4*>(dst) = w;
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

template <typename T, int D>
cudaError_t launch_packed_tc_variant(const PackedMaps& maps, const PackedParams& p,
                                     cudaStream_t stream) {
  auto kern = packed_tc_kernel<T, D>;
  static std::atomic<unsigned long long> attr_done{0};  // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(attr_done.load(std::memory_order_relaxed) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PackedLayout<D>::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const long long grid = static_cast<long long>(p.tiles) * p.Hkv;
  kern<<<static_cast<unsigned>(grid), kPackedThreads, PackedLayout<D>::SMEM_BYTES, stream>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace jvp
