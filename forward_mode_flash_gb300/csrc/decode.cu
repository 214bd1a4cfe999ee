// decode.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cached keys and joined.
//
// Per sequence b and query head h, over its n = lens[b] cached keys:
//   s_j = scale q . k_j,  o = sum_j exp(s_j - m) v_j / l,  lse = m + log l,
// with the running maximum m and sum l of an online softmax (fp32).
//
// Bound: memory.  Every cached row is read once by each block of query heads of
// its group (up to 16 on the tensor cores, 4 on the CUDA cores); nothing is
// reused beyond that, so what counts is bytes in flight: each warp keeps its own
// ring of row groups in shared memory, filled by 16-byte asynchronous copies some
// groups ahead, and no warp waits for another until the end of a segment.
// Measured with the join, in a CUDA graph: fp16, sequences of 131072 and 78806
// keys, 8 heads of 64: 68 us, 93 % of the copy rate; bf16, 48 of 18 to 4096 keys,
// 16/4 heads of 128: 41 us, 74 %; e4m3, 64 of 334 to 16384 keys, 16/2 heads of
// 128: 57.6 us, 70 % (5 us of the latter two are the join's latency, 2 to 3 the
// lookups in front of the first copies).
//
// Split: the work is the list of key tiles of all (sequence, key/value head,
// block of query heads) segments, in that order, and CTA c takes the c-th of
// `grid` equal ranges of it.  So CTAs are equally loaded whatever the
// lengths (which only the device knows), a captured launch follows lengths that
// change, and a CTA has at most two segments it shares with other CTAs.  A
// segment inside one CTA is written to the output at once; the others leave a
// normalised fp32 partial output and its log-sum-exp in the workspace, two
// slots per CTA, and the join kernel combines them in a fixed order (no
// atomics: results do not depend on timing).  Where no sequence can have more
// than a few tiles (a small block table), a CTA takes a whole segment and there
// is no second kernel.  (The host knows the table's width, not the lengths: 130
// keys, bf16, 16/4 heads of 128, take 5.2 us in a graph with a table of up to 16
// pages of 16, 6.8 us with any wider one.)  Parts are joined by log-sum-exps in
// fp32, so their shares are as exact as fp32 logits are.
//
// Tensor-core path (mma.sync m16n8k16): the products are formed transposed,
// S^T = K Q^T and O^T = V^T P^T, so that the 16 rows of the instruction are
// keys (or head-dimension columns) and its 8 columns the query heads of the
// group; each of a CTA's four warps takes 16 or 32 keys of a tile (8 KB of rows
// or less).  The order of the contraction index is free as long as both
// operands agree, so a lane's operand registers are whole 16-byte pieces of a
// cached row: for K the lane (g = lane / 4, t = lane % 4) holds pieces t,
// t + 4, ... of keys g and g + 8 and Q is permuted to match; for V it holds
// pieces g, g + 8, ... of keys 2t, 2t + 1, 2t + 8, 2t + 9, whose values are
// paired by key with byte permutes, and the permuted head-dimension order of
// O^T is undone at the store.  Pieces of a row are permuted in shared memory
// (K: by the row's lowest bit, V: by the next two) so that these reads hit
// distinct banks.  (tcgen05 wants 64 or more rows per product and its
// accumulator in TMEM; the tensor work here is a fraction of a per cent of its
// rate.)
//
// e4m3 caches: codes are converted to fp16 exactly.  The key scale 2^(ek-127)
// multiplies the logit.  The value scale goes into the exponent of the weight,
// w_j = 2^((x_j - m) + ev_j - 127 - mw) with its own running base mw (x_j the
// logit in log2 units), so no range of scales over- or underflows; the output
// is 2^mw sum w_j vc_j / l.  Queries become fp16 after a power-of-two
// normalisation per head (their largest magnitude to [2^14, 2^15)), so bf16
// queries of any magnitude keep their 8 bits.
//
// Rounding: the weights are rounded to 16 bits for the matrix product, fp16 ones
// scaled by 2^11 and with a maximum that moves past 2^4.9 (61148 at most): they
// keep their 11 bits down to 2^-25 of a row's largest and become 0 below 2^-36.
// (The base m - 11 of the exponents is kept as rounded, and compared by
// differences, so that large logits take no weight past its range.  bf16 weights
// need no scale; their maximum moves past 2^8.)  With a 16-bit cache the row sum
// adds the same rounded weights, so the output is the exact average under
// slightly perturbed weights; the log-sum-exp uses the unrounded sum.
#include <cmath>

#include "debug_checks.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace jvp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int tiles_of(int len, int tile) { return (len + tile - 1) / tile; }

// m16n8k16, fp32 accumulation, in place.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements held one 32-bit pair per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Elem<__half> {
  static constexpr bool kBF16 = false;
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr bool kBF16 = true;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float2 unpack2(uint32_t x, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// Largest over the eight lanes that share t = lane % 4.
__device__ __forceinline__ float max_over_g(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_g(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// ------------------------------------------------------------------ the split
// Total tiles of all sequences, and the sequence in which tile `want` of the
// list (for want in range) lies, with the tiles before it.  Executed by the
// whole block; every thread gets the same answer.  Each thread sums a run of
// B / blockDim sequences.
struct Place {
  long long total, before;
  int b;
};
template <int THREADS>
__device__ __forceinline__ long long block_exclusive(long long x, long long* total,
                                                     long long* sh /* THREADS / 32 */) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  long long base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += sh[w];
    all += sh[w];
  }
  *total = all;
  return base + incl - x;
}

struct SplitShared {
  long long scan[kWarps];
  Place place;
};

// A CTA's part of one segment: keys of tiles [t0, t1) of sequence b for
// key/value head hk and block hb of its query heads.  slot: where its partial
// output goes (-1: it is the whole segment).
struct Piece {
  int b, hk, hb, len, t0, t1, slot;
  long long first;  // the segment's first tile in the list, and its tiles
  int nt;
};

// This CTA's range of the list, segment by segment.
template <int TILE>
struct Walker {
  long long at, hi, seq_first, HH, W, G;  // W tiles in all, on G CTAs
  int b, len, nt;

  // False: nothing to do here.  Executed by the whole block.
  __device__ __forceinline__ bool start(const DecodeParams& p, SplitShared* sh) {
    const PagedCache& c = p.c;
    HH = static_cast<long long>(c.Hkv) * p.head_blocks;
    bool bad = false;
    if (p.direct) {  // one segment per CTA, with or without keys
      at = blockIdx.x, hi = at + 1, seq_first = 0;
      b = static_cast<int>(at / HH);
      len = clamp_len(c, __ldg(p.lens + b), &bad), nt = tiles_of(len, TILE);
      if (bad && at % HH == 0 && threadIdx.x == 0) atomicOr(c.status, kStatusIndex);
      return true;
    }
    const int per = (c.B + kThreads - 1) / kThreads;  // sequences per thread
    const int b_lo = min(c.B, static_cast<int>(threadIdx.x) * per), b_hi = min(c.B, b_lo + per);
    long long mine = 0;
    for (int i = b_lo; i < b_hi; ++i) mine += tiles_of(clamp_len(c, __ldg(p.lens + i), &bad), TILE);
    long long seq_total;
    const long long before = block_exclusive<kThreads>(mine, &seq_total, sh->scan);
    W = seq_total * HH;
    G = min(static_cast<long long>(p.grid), W);
    if (static_cast<long long>(blockIdx.x) >= G) return false;
    at = W * blockIdx.x / G, hi = W * (blockIdx.x + 1) / G;
    // the thread whose run of sequences holds tile `at` finds the sequence
    if (at >= before * HH && at < (before + mine) * HH) {
      long long first = before;
      int i = b_lo;
      for (; i < b_hi; ++i) {
        const int t = tiles_of(clamp_len(c, __ldg(p.lens + i), &bad), TILE);
        if (at < (first + t) * HH) break;
        first += t;
      }
      sh->place.b = i;
      sh->place.before = first;
    }
    __syncthreads();
    b = sh->place.b;
    seq_first = sh->place.before * HH;
    len = clamp_len(c, __ldg(p.lens + b), &bad), nt = tiles_of(len, TILE);
    return true;
  }
  __device__ __forceinline__ bool next(const DecodeParams& p, Piece* s) {
    if (at >= hi) return false;
    if (p.direct) {
      const int seg = static_cast<int>(at % HH);
      s->hk = seg / p.head_blocks, s->hb = seg % p.head_blocks;
      s->b = b, s->len = len, s->t0 = 0, s->t1 = nt, s->slot = -1;
      at = hi;
      return true;
    }
    bool bad = false;
    while (at >= seq_first + nt * HH) {  // next sequence with keys (at < hi <= W: there is one)
      seq_first += nt * HH;
      ++b;
      len = clamp_len(p.c, __ldg(p.lens + b), &bad), nt = tiles_of(len, TILE);
    }
    const int seg = static_cast<int>((at - seq_first) / nt);
    s->hk = seg / p.head_blocks, s->hb = seg % p.head_blocks;
    const long long first = seq_first + static_cast<long long>(seg) * nt;
    s->b = b, s->len = len;
    s->t0 = static_cast<int>(at - first);
    s->t1 = static_cast<int>(min(hi - first, static_cast<long long>(nt)));
    s->slot = (s->t0 == 0 && s->t1 == nt) ? -1 : (s->t0 > 0 ? 0 : 1);
    s->first = first, s->nt = nt;
    at = first + s->t1;
    return true;
  }
  // For the join, by the CTA that begins a segment: the CTAs that share it
  // (CTA c holds tiles [W c / G, W (c + 1) / G); this one is the first).
  __device__ __forceinline__ void note(const DecodeParams& p, const Piece& s) const {
    if (p.direct || s.t0 > 0 || threadIdx.x != 0) return;
    const int c1 = static_cast<int>(((s.first + s.nt) * G - 1) / W);
    if (JVP_CHECK(s.b < p.c.B && s.hk < p.c.Hkv && s.hb < p.head_blocks && c1 < p.grid, p.c.status,
                  kChkGlobalRow))
      p.ws_cta[(static_cast<long long>(s.b) * p.c.Hkv + s.hk) * p.head_blocks + s.hb] =
          make_int2(static_cast<int>(blockIdx.x), c1);
  }
};

// Slot of a partial output: log-sum-exp (log2 units) per head, and a row of
// ws_ld floats per head.
__device__ __forceinline__ long long slot_row(const DecodeParams& p, long long cta, int slot,
                                              int hpb, int h) {
  return (cta * 2 + slot) * hpb + h;
}

// ------------------------------------------------------------------ tensor cores
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool on) {
  // copies 16 bytes, or writes 16 zero bytes and reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ld_shared(uint32_t a, uint32_t (&x)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ld_shared(uint32_t a, uint32_t (&x)[2]) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(a) : "memory");
}

// The ring of one warp: ST groups of KT keys, K rows then V rows.
template <int DPAD, bool E4M3>
struct Ring {
  static constexpr int ROWB = DPAD * (E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int KT = decode_warp_keys(DPAD, E4M3);
  static constexpr int PIECES = ROWB / 16;
  static constexpr int STAGE = 2 * KT * ROWB;
  static constexpr int ST = decode_stages(E4M3);
  static constexpr int WARP = ST * STAGE;
  // byte offset of 16-byte piece x of a row
  static __device__ __forceinline__ int k_at(int row, int x) {
    return row * ROWB + ((PIECES >= 8 ? x ^ ((row & 1) << 2) : x) << 4);
  }
  static __device__ __forceinline__ int v_at(int row, int x) {
    return KT * ROWB + row * ROWB + ((PIECES >= 8 ? x ^ (row & 6) : x ^ ((row >> 1) & 3)) << 4);
  }
};

// A warp's state in shared memory: accumulator fragments, and (m, mw, l, lx) of
// heads 2t, 2t + 1 (+ 8 n).
template <int DPAD, int NG>
struct Exchange {
  float4 acc[NG * DPAD / 16][32];
  float4 stat[NG * 2][4];
};

// TQ: type of q and o, and of a 16-bit cache.  NG: groups of 8 query heads.
template <typename TQ, int DPAD, bool E4M3, int NG>
__global__ void __launch_bounds__(kThreads, decode_ctas_per_sm(DPAD, NG, E4M3))
    decode_tc_kernel(const DecodeParams p) {
  using R = Ring<DPAD, E4M3>;
  constexpr int HPB = 8 * NG;
  constexpr int KT = R::KT, RG = KT / 16, TILE = kWarps * KT, ST = R::ST;
  static_assert(ST == 2 || !E4M3, "scale bytes are held for one group ahead");
  constexpr bool kBF16 = Elem<TQ>::kBF16 && !E4M3;  // operand type of the products
  // weights are 2^(x - base), the base kShift below a maximum; it moves where they
  // would pass 2^kTop
  constexpr float kShift = kBF16 ? 0.f : 11.f, kUnshift = kBF16 ? 1.f : 1.f / 2048.f;
  constexpr float kTop = kBF16 ? 8.f : 15.9f;
  // (the maximum itself where a step of fp32 is 16, so that m - 11 would be m - 16)
  auto base = [&](float m) { return m - (m - kShift) > kTop ? m : m - kShift; };
  constexpr int KS = DPAD / 16;                     // contraction steps of S^T
  constexpr int EPC = E4M3 ? 16 : 8;                // elements of a 16-byte piece
  constexpr int KSP = EPC / 4;                      // contraction steps per K piece
  constexpr int KP = DPAD / (4 * EPC);              // K pieces per lane and key
  constexpr int MT = DPAD / 16;                     // 16-column tiles of O^T
  constexpr int VW = E4M3 ? DPAD / 32 : 4;          // 32-bit words of a V piece (8 lanes a row)
  constexpr int VP = E4M3 ? 1 : DPAD / 64;          // V pieces per lane and key
  constexpr int VE = E4M3 ? DPAD / 8 : 8;           // elements of a V piece
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using X = Exchange<DPAD, NG>;
  auto* sh = reinterpret_cast<SplitShared*>(smem_raw);
  X* xch = reinterpret_cast<X*>(smem_raw + 128);  // two warps' states
  static_assert(sizeof(SplitShared) <= 128, "shared memory layout");
  const PagedCache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem_raw + 128 + 2 * sizeof(X)) + warp * R::WARP;
  const int D = c.D;
  using TC = typename std::conditional<E4M3, uint8_t, TQ>::type;
  const TC* kc = static_cast<const TC*>(c.k);
  const TC* vc = static_cast<const TC*>(c.v);
  // every aligned run of 16 keys lies in one page
  const bool runs = c.page_size % 16 == 0;
  // this lane's part of a group's copies: piece x of rows lr, lr + RS, ...
  constexpr int RS = 32 / R::PIECES, NCP = KT / RS;
  const int lr = lane / R::PIECES, x = lane % R::PIECES;
  const bool col_on = x * EPC < D;
  const int xcol = col_on ? x * EPC : 0;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walker<TILE> walker;
  if (!walker.start(p, sh)) return;
  Piece s;  // the piece whose groups are being copied
  walker.next(p, &s);

  auto first_key = [&](int it) { return (s.t0 + it) * TILE + warp * KT; };
  // Block-table entry of this lane's key of group it (its 16-key run's first
  // key where runs lie in one page), unchecked, and that key's row of the
  // page.  Loaded a group ahead of the copies that need it.
  int raw = -1, row = 0;
  bool looked = false;
  auto look_up = [&](int it) {
    const int j = first_key(it) + (runs ? (KT == 32 ? lane & 16 : 0) : lane);
    looked = it < s.t1 - s.t0 && (runs || lane < KT) && j < s.len;
    if (looked) {
      int entry;
      split_position(c, j, &entry, &row);
      raw = __ldg(c.table + s.b * c.table_stride + entry);
    }
  };
  // Starts the copies of group it (whose entries have been looked up) into
  // its stage; e4m3: also loads the scale bytes of key `lane` (K low, V high
  // byte).  keep_next: keys of the group that exist and whose page does.
  unsigned sb_next = 0;
  uint32_t keep_next = 0, keeps[ST - 1];  // of the group issued last; of the groups in flight
  auto issue = [&](int it) {
    const int j0 = first_key(it);
    if (it < s.t1 - s.t0 && j0 < s.len) {
      const bool have = looked && raw >= 0 && raw < c.pages;
      if (looked && !have) atomicOr(c.status, kStatusIndex);
      const int left = s.len - j0;
      keep_next = __ballot_sync(0xffffffffu, have) & (KT == 32 ? 0xFFFFFFFFu : 0xFFFFu) &
                  (left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u);
      const int page = have ? raw : 0, r0 = have ? row : 0;
      const TC* kp = kc + page * c.sk.b + s.hk * c.sk.h + r0 * c.sk.n;
      const TC* vp = vc + page * c.sv.b + s.hk * c.sv.h + r0 * c.sv.n;
      if (E4M3 && ((keep_next >> lane) & 1u)) {
        const long long at = (static_cast<long long>(page) * c.Hkv + s.hk) * c.page_size + r0 +
                             (runs ? lane & 15 : 0);
        sb_next = __ldg(c.k_scale + at) | (static_cast<unsigned>(__ldg(c.v_scale + at)) << 8);
      }
      const uint32_t dst = ring + (it % ST) * R::STAGE;
      if (runs) {
        // (the pointers of run h of the group are lane 16 h's)
#pragma unroll
        for (int h = 0; h < RG; ++h) {
          const TC* kr = reinterpret_cast<const TC*>(__shfl_sync(
                             0xffffffffu, reinterpret_cast<unsigned long long>(kp), 16 * h)) +
                         lr * c.sk.n + xcol;
          const TC* vr = reinterpret_cast<const TC*>(__shfl_sync(
                             0xffffffffu, reinterpret_cast<unsigned long long>(vp), 16 * h)) +
                         lr * c.sv.n + xcol;
          const uint32_t keep = (keep_next >> (16 * h)) & 0xFFFFu;
#pragma unroll
          for (int i = 0; i < 16 / RS; ++i) {
            const int r = 16 * h + i * RS + lr;
            const bool on = col_on && (keep == 0xFFFFu || ((keep >> (i * RS + lr)) & 1u));
            if (!JVP_CHECK(R::v_at(r, x) + 16 <= R::STAGE, c.status, kChkSmem)) continue;
            copy_async16(dst + R::k_at(r, x), kr, on);
            copy_async16(dst + R::v_at(r, x), vr, on);
            kr += RS * c.sk.n, vr += RS * c.sv.n;
          }
        }
      } else {
#pragma unroll 4
        for (int i = 0; i < NCP; ++i) {
          const int r = i * RS + lr;
          const TC* kr = reinterpret_cast<const TC*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kp), r));
          const TC* vr = reinterpret_cast<const TC*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vp), r));
          const bool on = col_on && ((keep_next >> r) & 1u);
          if (!JVP_CHECK(R::v_at(r, x) + 16 <= R::STAGE, c.status, kChkSmem)) continue;
          copy_async16(dst + R::k_at(r, x), kr + xcol, on);
          copy_async16(dst + R::v_at(r, x), vr + xcol, on);
        }
      }
    }
    copy_async_commit();
  };
  uint32_t qf[NG][KS][2];
  float qs[NG][2];
  // The first groups of piece s on their way, and its query operand.
  auto begin = [&]() {
    __syncwarp();  // the ring has been read
#pragma unroll
    for (int it = 0; it < ST - 1; ++it) {
      look_up(it);
      issue(it);
      keeps[it] = keep_next;
    }
    look_up(ST - 1);
    const int h0 = s.hk * p.group + s.hb * HPB;
    const int nh = min(HPB, p.group - s.hb * HPB);
    // ---- Q^T operand: lane (g, t) holds head g (+ 8 n), permuted to match K
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int h = n * 8 + g;
      const TQ* q = static_cast<const TQ*>(p.q) + s.b * p.sq.b + (h0 + h) * p.sq.h;
      float x[KS][4];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int d = (t + 4 * (ks / KSP)) * EPC + 4 * (ks % KSP);
        uint2 w = make_uint2(0, 0);
        if (h < nh && d < D) w = __ldg(reinterpret_cast<const uint2*>(q + d));
        if constexpr (E4M3) {
          const float2 a = unpack2(w.x, Elem<TQ>::kBF16), b = unpack2(w.y, Elem<TQ>::kBF16);
          x[ks][0] = a.x, x[ks][1] = a.y, x[ks][2] = b.x, x[ks][3] = b.y;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[ks][i]));
        } else {
          qf[n][ks][0] = w.x, qf[n][ks][1] = w.y;
        }
      }
      if constexpr (E4M3) {
        // q * 2^-eq with the largest magnitude in [2^14, 2^15) (an exponent
        // outside [-126, 126] is clamped: such a head's logits are 0 or huge)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;  // eq
        const int ec = max(-126, min(126, e));
        const float down = __uint_as_float(static_cast<unsigned>(127 - ec) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[n][ks][0] = pack2(x[ks][0] * down, x[ks][1] * down, false);
          qf[n][ks][1] = pack2(x[ks][2] * down, x[ks][3] * down, false);
        }
        // (of the head that this lane loads; lane 4 h has head h's)
        const float f = p.scale_log2 * __uint_as_float(static_cast<unsigned>(127 + ec) << 23);
        qs[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        qs[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      } else {
        qs[n][0] = qs[n][1] = p.scale_log2;
      }
    }
  };

  begin();
  while (true) {
    float m[NG][2], mw[NG][2], l[NG][2], lx[NG][2], acc[NG][MT][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[n][i] = mw[n][i] = -INFINITY, l[n][i] = lx[n][i] = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][mt][i] = 0.f;
    }

    for (int it = 0; it < s.t1 - s.t0 && first_key(it) < s.len; ++it) {
      copy_async_wait<ST - 2>();
      __syncwarp();  // every lane's copies of group it are in; group it - 1 has been read
      const unsigned sb = sb_next;
      const uint32_t keep = keeps[0];
      issue(it + ST - 1);
      look_up(it + ST);
#pragma unroll
      for (int i = 0; i + 1 < ST - 1; ++i) keeps[i] = keeps[i + 1];
      keeps[ST - 2] = keep_next;
      auto kept = [&](int i) -> bool { return (keep >> i) & 1u; };
      const uint32_t st = ring + (it % ST) * R::STAGE;

      // ---- S^T = K Q^T
      float sc[RG][NG][4];
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[rg][n][i] = 0.f;
#pragma unroll
        for (int u = 0; u < KP; ++u) {
          uint32_t w[2][4];  // piece t + 4u of keys g and g + 8
          ld_shared(st + R::k_at(rg * 16 + g, t + 4 * u), w[0]);
          ld_shared(st + R::k_at(rg * 16 + g + 8, t + 4 * u), w[1]);
#pragma unroll
          for (int k = 0; k < KSP; ++k) {
            uint32_t a[4];  // (key g, lo), (key g + 8, lo), (key g, hi), (key g + 8, hi)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (E4M3) {
                e4m3x4_to_half2x2(w[r][k], a[r], a[2 + r]);
              } else {
                a[r] = w[r][2 * k];
                a[2 + r] = w[r][2 * k + 1];
              }
            }
#pragma unroll
            for (int n = 0; n < NG; ++n)
              mma16816<kBF16>(sc[rg][n], a[0], a[1], a[2], a[3], qf[n][u * KSP + k][0],
                              qf[n][u * KSP + k][1]);
          }
        }
      }
      // scales of this lane's keys g + 8 r
      float kscale[2 * RG], vexp[2 * RG];
      if constexpr (E4M3) {
#pragma unroll
        for (int r = 0; r < 2 * RG; ++r) {
          const unsigned x = __shfl_sync(0xffffffffu, sb, g + 8 * r);
          kscale[r] = scale_value(x & 0xFFu);
          vexp[r] = static_cast<float>(static_cast<int>(x >> 8) - 127);
        }
      }
      // ---- logits in log2 units, weights
      uint32_t pf[RG][NG][2];  // P^T operand: keys 2t, 2t + 1 (and + 8) of head g
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float x[2 * RG][2], pw[2 * RG][2];  // [key g + 8 r][head 2t + i]
        // The bases of the exponents move only where a weight would pass 2^kTop
        // (ratios are exact for any base): one vote, and the reductions over
        // the keys only then.  (Over e4m3 m is the base of the row sum, which
        // is fp32, and mw that of the weights, relative to m: beside a large
        // logit fp32 would not hold a value's exponent.  Else m is both.)
        bool need = false;
#pragma unroll
        for (int r = 0; r < 2 * RG; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = sc[r / 2][n][2 * (r & 1) + i] * (E4M3 ? kscale[r] * qs[n][i] : qs[n][i]);
            x[r][i] = kept(g + 8 * r) ? y : -INFINITY;
            const float above = x[r][i] - m[n][i];
            need |= above > (E4M3 ? 8.f : kTop);
            if constexpr (E4M3) need |= above + (vexp[r] - mw[n][i]) > kTop;
          }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2 * RG; ++r) top = fmaxf(top, x[r][i]);
            top = max_over_g(top);
            const float m_new = fmaxf(m[n][i], E4M3 ? top : base(top));
            const float move = m_new == m[n][i] ? 0.f : m[n][i] - m_new;
            float a = exp2f(move);
            m[n][i] = m_new;
            l[n][i] *= a, lx[n][i] *= a;
            if constexpr (E4M3) {
              float topw = -INFINITY;
#pragma unroll
              for (int r = 0; r < 2 * RG; ++r) topw = fmaxf(topw, (x[r][i] - m_new) + vexp[r]);
              const float mw_old = mw[n][i] + move;
              const float mw_new = fmaxf(mw_old, base(max_over_g(topw)));
              a = mw_new == mw_old ? 1.f : exp2f(mw_old - mw_new);
              mw[n][i] = mw_new;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[n][mt][i] *= a;
              acc[n][mt][2 + i] *= a;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mu = m[n][i] == -INFINITY ? 0.f : m[n][i];
          const float mwu = mw[n][i] == -INFINITY ? 0.f : mw[n][i];
#pragma unroll
          for (int r = 0; r < 2 * RG; ++r) {
            if constexpr (E4M3) {
              l[n][i] += ex2_approx(x[r][i] - mu);
              pw[r][i] = ex2_approx((x[r][i] - mu) + (vexp[r] - mwu));
            } else {
              pw[r][i] = ex2_approx(x[r][i] - mu);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 2 * RG; ++r) {
          const uint32_t w = pack2(pw[r][0], pw[r][1], kBF16);
          if constexpr (!E4M3) {  // sums of the rounded and the unrounded weights
            const float2 f = unpack2(w, kBF16);
            l[n][0] += f.x, l[n][1] += f.y;
            lx[n][0] += pw[r][0], lx[n][1] += pw[r][1];
          }
          pf[r / 2][n][r & 1] = transpose8x8(w);
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
#pragma unroll
        for (int u = 0; u < VP; ++u) {
          uint32_t vf[4][VW];  // piece g + 8u of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = rg * 16 + 2 * t + (r & 1) + 8 * (r >> 1);
            if constexpr (VW == 4) ld_shared(st + R::v_at(row, g + 8 * u), vf[r]);
            else ld_shared(st + R::v_at(row, g >> 1) + 8 * (g & 1), vf[r]);
          }
#pragma unroll
          for (int k = 0; k < MT / VP; ++k) {
            const int mt = u * (MT / VP) + k;
            uint32_t a[4];  // (column a, keys 2t, 2t+1), (column b, ..), (a, keys + 8), (b, ..)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (E4M3) {
                const uint32_t w =
                    __byte_perm(vf[2 * r][k / 2], vf[2 * r + 1][k / 2], (k & 1) ? 0x7362 : 0x5140);
                e4m3x4_to_half2x2(w, a[2 * r], a[2 * r + 1]);
              } else {
                a[2 * r] = __byte_perm(vf[2 * r][k], vf[2 * r + 1][k], 0x5410);
                a[2 * r + 1] = __byte_perm(vf[2 * r][k], vf[2 * r + 1][k], 0x7632);
              }
            }
#pragma unroll
            for (int n = 0; n < NG; ++n)
              mma16816<kBF16>(acc[n][mt], a[0], a[1], a[2], a[3], pf[rg][n][0], pf[rg][n][1]);
          }
        }
      }
    }

    // ---- the next piece's first groups, then the join of the four warps
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] = sum_over_g(l[n][i]);
        lx[n][i] = E4M3 ? l[n][i] : sum_over_g(lx[n][i]);
      }
    walker.note(p, s);
    const Piece done = s;
    const bool more = walker.next(p, &s);
    if (more) begin();
    auto put = [&](X& to) {
#pragma unroll
      for (int n = 0; n < NG; ++n) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          to.acc[n * MT + mt][lane] =
              make_float4(acc[n][mt][0], acc[n][mt][1], acc[n][mt][2], acc[n][mt][3]);
        if (g == 0)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            to.stat[n * 2 + i][t] = make_float4(m[n][i], mw[n][i], l[n][i], lx[n][i]);
      }
    };
    // merge of another warp's state into this one's, each relative to its own
    // maxima
    auto take = [&](const X& from) {
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float own[2], oth[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 st = from.stat[n * 2 + i][t];
          const float mine = m[n][i], M = fmaxf(mine, st.x), mu = M == -INFINITY ? 0.f : M;
          const float a = exp2f(mine - mu), b = exp2f(st.x - mu);
          l[n][i] = a * l[n][i] + b * st.z;
          lx[n][i] = a * lx[n][i] + b * st.w;
          m[n][i] = M;
          own[i] = a, oth[i] = b;
          if constexpr (E4M3) {
            const float u = mw[n][i] + (mine - mu), v = st.y + (st.x - mu);
            const float W = fmaxf(u, v), wu = W == -INFINITY ? 0.f : W;
            own[i] = exp2f(u - wu), oth[i] = exp2f(v - wu);
            mw[n][i] = W;
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float4 o = from.acc[n * MT + mt][lane];
          acc[n][mt][0] = own[0] * acc[n][mt][0] + oth[0] * o.x;
          acc[n][mt][1] = own[1] * acc[n][mt][1] + oth[1] * o.y;
          acc[n][mt][2] = own[0] * acc[n][mt][2] + oth[0] * o.z;
          acc[n][mt][3] = own[1] * acc[n][mt][3] + oth[1] * o.w;
        }
      }
    };
    __syncthreads();  // the last join has been read
    if (warp >= 2) put(xch[warp - 2]);
    __syncthreads();
    if (warp < 2) take(xch[warp]);
    if (warp == 1) put(xch[1]);  // (only this warp read it)
    __syncthreads();
    if (warp == 0) {
      take(xch[1]);
      const int h0 = done.hk * p.group + done.hb * HPB;
      const int nh = min(HPB, p.group - done.hb * HPB);
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = n * 8 + 2 * t + i;
          if (h >= nh) continue;
          const float mu = m[n][i] == -INFINITY ? 0.f : m[n][i];
          // (l may be NaN: a NaN among the logits reaches every output of the
          // row.  With a 16-bit cache l and the accumulator have the same
          // base.)
          float f = l[n][i] == 0.f ? 0.f : 1.f / l[n][i];
          if (E4M3) f *= exp2f(mw[n][i]);  // (0 without keys)
          const float lse = lx[n][i] == 0.f ? -INFINITY
                            : E4M3          ? mu + log2f(lx[n][i])
                                            : mu + kShift + log2f(lx[n][i] * kUnshift);
          const long long ws = slot_row(p, blockIdx.x, done.slot, HPB, h);
          if (!JVP_CHECK(done.slot >= 0 ? ws < 2ll * p.grid * HPB : done.b < c.B && h0 + h < p.H,
                         c.status, kChkGlobalRow))
            continue;
          if (g == 0) {
            if (done.slot >= 0) p.ws_lse[ws] = lse;
            else if (p.lse) p.lse[static_cast<long long>(done.b) * p.H + h0 + h] = lse * 0.6931471805599453f;
          }
#pragma unroll
          for (int u = 0; u < MT / 4; ++u) {  // eight columns from d
            const int d = E4M3 ? g * VE + 8 * u : (g + 8 * u) * 8;
            if (d >= D || !JVP_CHECK(d + 8 <= D, c.status, kChkGlobalCol)) continue;
            float o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = acc[n][4 * u + k][i] * f;
              o[2 * k + 1] = acc[n][4 * u + k][2 + i] * f;
            }
            if (done.slot >= 0) {
              float4* dst = reinterpret_cast<float4*>(p.ws_o + ws * DPAD + d);
              dst[0] = make_float4(o[0], o[1], o[2], o[3]);
              dst[1] = make_float4(o[4], o[5], o[6], o[7]);
            } else {
              TQ* dst = static_cast<TQ*>(p.o) + done.b * p.so.b + (h0 + h) * p.so.h + d;
              if (p.o_vec) {
                *reinterpret_cast<uint4*>(dst) =
                    make_uint4(pack2(o[0], o[1], Elem<TQ>::kBF16), pack2(o[2], o[3], Elem<TQ>::kBF16),
                               pack2(o[4], o[5], Elem<TQ>::kBF16), pack2(o[6], o[7], Elem<TQ>::kBF16));
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = Elem<TQ>::put(o[k]);
              }
            }
          }
        }
    }
    if (!more) break;
  }
}

// ------------------------------------------------------------------ CUDA cores
// Any type and alignment: fp32 arithmetic.  DPAD / 16 lanes share a key (lane t
// of them takes the columns 4 (t + LK u) .. + 3), so a warp takes 8 or 4 keys at
// once; it loads the next ones' rows before it works on these.  A CTA takes HPB
// query heads, each lane summing its own keys' weighted values until the end of
// the piece.  Measured in a CUDA graph, fp32 caches: 60000 keys of 8 ungrouped
// heads of 128 in 79 us, 91 % of the copy rate (four CTAs per SM; three: 90 %); 16
// sequences of 500 to 4000 keys, 8 heads on 2 of 128, 28 us, 46 % (three; four, of
// 128 registers a thread: 34 us).  The latter has some ten rounds a warp, each
// waiting for rows that were asked for one round ahead, and a start and a join;
// its FMAs are 2 us.  bf16, 48 of 4000 keys, 16/4 heads: rows of 100, 115 us, 39 %;
// rows of 128 off their 16-byte alignment (single loads), 277 us, 21 %.
template <typename T>
struct Raw {  // four columns as stored
  uint32_t w[sizeof(T)];
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load4(const T* row, int d, int D) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) r.w[i] = 0u;
  if constexpr (VEC) {
    if (d < D) {
      if constexpr (sizeof(T) == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + d));
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
      } else if constexpr (sizeof(T) == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(row + d));
        r.w[0] = x.x, r.w[1] = x.y;
      } else {
        r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + d));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < D) {
        if constexpr (sizeof(T) == 4)
          r.w[i] = __ldg(reinterpret_cast<const uint32_t*>(row) + d + i);
        else if constexpr (sizeof(T) == 2)
          r.w[i / 2] |= static_cast<uint32_t>(
                            __ldg(reinterpret_cast<const unsigned short*>(row) + d + i))
                        << (16 * (i & 1));
        else
          r.w[0] |= static_cast<uint32_t>(__ldg(row + d + i)) << (8 * i);
      }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ float4 value4(const Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
    return make_float4(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]), __uint_as_float(r.w[2]),
                       __uint_as_float(r.w[3]));
  } else if constexpr (sizeof(T) == 2) {
    const float2 a = unpack2(r.w[0], Elem<T>::kBF16), b = unpack2(r.w[1], Elem<T>::kBF16);
    return make_float4(a.x, a.y, b.x, b.y);
  } else {
    uint32_t a, b;
    e4m3x4_to_half2x2(r.w[0], a, b);
    const float2 fa = unpack2(a, false), fb = unpack2(b, false);
    return make_float4(fa.x, fa.y, fb.x, fb.y);
  }
}

template <int HPB, int DPAD>
struct SimtShared {
  SplitShared split;
  float m[kWarps][HPB], l[kWarps][HPB];
  alignas(16) float q[HPB][DPAD];
  alignas(16) float acc[kWarps][HPB][DPAD];
};

template <typename TQ, int DPAD, bool E4M3, int HPB, bool VEC>
__global__ void __launch_bounds__(kThreads, decode_simt_ctas_per_sm(HPB))
decode_simt_kernel(const DecodeParams p) {
  constexpr int LK = DPAD / 16, NC = 4, KR = 32 / LK;  // lanes of a key, pieces of a lane, keys
  constexpr int TILE = kDecodeSimtTile, KT = TILE / kWarps, R = KT / KR;
  static_assert(KT == 16 && R * KR == KT, "rounds of a warp's part of a tile");
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto* sh = reinterpret_cast<SimtShared<HPB, DPAD>*>(smem_raw);
  const PagedCache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / LK, t = lane % LK;
  const int D = c.D;
  using TC = typename std::conditional<E4M3, uint8_t, TQ>::type;
  const TC* kc = static_cast<const TC*>(c.k);
  const TC* vc = static_cast<const TC*>(c.v);
  auto over_keys = [&](float x, auto op) {  // over the lanes with this t
#pragma unroll
    for (int o = LK; o < 32; o <<= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  auto add = [](float x, float y) { return x + y; };
  auto larger = [](float x, float y) { return fmaxf(x, y); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walker<TILE> walker;
  if (!walker.start(p, &sh->split)) return;
  Piece s;
  while (walker.next(p, &s)) {
    const int h0 = s.hk * p.group + s.hb * HPB;
    const int nh = min(HPB, p.group - s.hb * HPB);
    __syncthreads();
    for (int e = threadIdx.x; e < HPB * DPAD; e += kThreads) {
      const int h = e / DPAD, d = e % DPAD;
      sh->q[h][d] = (h < nh && d < D)
                     ? Elem<TQ>::get(static_cast<const TQ*>(p.q)[s.b * p.sq.b + (h0 + h) * p.sq.h + d])
                     : 0.f;
    }
    __syncthreads();
    float m[HPB], l[HPB];
    float4 acc[HPB][NC];
#pragma unroll
    for (int h = 0; h < HPB; ++h) {
      m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
      for (int u = 0; u < NC; ++u) acc[h][u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // Rounds i of the piece: a key's page is looked up a round before its rows
    // are asked for, its K row during the second half of the round before (when
    // the last one's scores are formed), its V row at the end of that round.
    const int rounds = (s.t1 - s.t0) * R;
    long long ko = 0, vo = 0, so = 0;  // of the next round's key
    bool next_on = false;
    auto look_up = [&](int i) {
      next_on = false;
      if (i >= rounds) return;
      const int j = (s.t0 + i / R) * TILE + warp * KT + (i % R) * KR + g;
      if (j >= s.len) return;
      int entry, row;
      split_position(c, j, &entry, &row);
      const int page = page_of(c, s.b, entry);
      if (page < 0) return;
      next_on = true;
      ko = page * c.sk.b + s.hk * c.sk.h + row * c.sk.n;
      vo = page * c.sv.b + s.hk * c.sv.h + row * c.sv.n;
      if (E4M3) so = (static_cast<long long>(page) * c.Hkv + s.hk) * c.page_size + row;
    };
    Raw<TC> k[NC], v[NC];
    unsigned ke = 127u, ve = 127u;
    auto fetch = [&](Raw<TC>(&x)[NC], const TC* row, const uint8_t* scale, unsigned* byte) {
      const int width = next_on ? D : 0;
#pragma unroll
      for (int u = 0; u < NC; ++u) x[u] = load4<TC, VEC>(row, 4 * (t + LK * u), width);
      if (E4M3) *byte = next_on ? __ldg(scale + so) : 127u;
    };
    look_up(0);
    fetch(k, kc + ko, c.k_scale, &ke);
    fetch(v, vc + vo, c.v_scale, &ve);
    bool on = next_on;
    look_up(1);
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
      float w[HPB];
      bool need = false;
      const float ks = E4M3 ? p.scale_log2 * scale_value(ke) : p.scale_log2;
#pragma unroll
      for (int h = 0; h < HPB; ++h) w[h] = 0.f;
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const float4 x = value4<TC>(k[u]);
#pragma unroll
        for (int h = 0; h < HPB; ++h) {
          const float4 q = *reinterpret_cast<const float4*>(&sh->q[h][4 * (t + LK * u)]);
          w[h] = fmaf(x.x, q.x, fmaf(x.y, q.y, fmaf(x.z, q.z, fmaf(x.w, q.w, w[h]))));
        }
      }
      fetch(k, kc + ko, c.k_scale, &ke);
#pragma unroll
      for (int h = 0; h < HPB; ++h) {
#pragma unroll
        for (int o = 1; o < LK; o <<= 1) w[h] += __shfl_xor_sync(0xffffffffu, w[h], o);
        w[h] = on ? w[h] * ks : -INFINITY;
        need |= w[h] > m[h] + 8.f;
      }
      if (__any_sync(0xffffffffu, need)) {  // (as on the tensor cores)
#pragma unroll
        for (int h = 0; h < HPB; ++h) {
          const float m_new = fmaxf(m[h], over_keys(w[h], larger));
          const float a = m_new == m[h] ? 1.f : exp2f(m[h] - m_new);
          m[h] = m_new;
          l[h] *= a;
#pragma unroll
          for (int u = 0; u < NC; ++u)
            acc[h][u].x *= a, acc[h][u].y *= a, acc[h][u].z *= a, acc[h][u].w *= a;
        }
      }
      const float vs = E4M3 ? scale_value(ve) : 1.f;
#pragma unroll
      for (int h = 0; h < HPB; ++h) {
        w[h] = exp2f(w[h] - (m[h] == -INFINITY ? 0.f : m[h]));
        l[h] += w[h];
        if (E4M3) w[h] *= vs;
      }
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const float4 x = value4<TC>(v[u]);
#pragma unroll
        for (int h = 0; h < HPB; ++h) {
          acc[h][u].x = fmaf(w[h], x.x, acc[h][u].x);
          acc[h][u].y = fmaf(w[h], x.y, acc[h][u].y);
          acc[h][u].z = fmaf(w[h], x.z, acc[h][u].z);
          acc[h][u].w = fmaf(w[h], x.w, acc[h][u].w);
        }
      }
      fetch(v, vc + vo, c.v_scale, &ve);
      on = next_on;
      look_up(i + 2);
    }
#pragma unroll
    for (int h = 0; h < HPB; ++h) {
      const float ls = over_keys(l[h], add);
      if (lane == 0) sh->m[warp][h] = m[h], sh->l[warp][h] = ls;
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const float4 a =
            make_float4(over_keys(acc[h][u].x, add), over_keys(acc[h][u].y, add),
                        over_keys(acc[h][u].z, add), over_keys(acc[h][u].w, add));
        if (g == 0) *reinterpret_cast<float4*>(&sh->acc[warp][h][4 * (t + LK * u)]) = a;
      }
    }
    walker.note(p, s);
    __syncthreads();
    for (int e = threadIdx.x; e < nh * DPAD; e += kThreads) {
      const int h = e / DPAD, d = e % DPAD;
      if (d >= D) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh->m[w][h]);
      const float mu = M == -INFINITY ? 0.f : M;
      float sum = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = exp2f(sh->m[w][h] - mu);
        sum += a * sh->l[w][h];
        o += a * sh->acc[w][h][d];
      }
      o *= sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : mu + log2f(sum);
      if (s.slot >= 0) {
        const long long ws = slot_row(p, blockIdx.x, s.slot, HPB, h);
        p.ws_o[ws * DPAD + d] = o;
        if (d == 0) p.ws_lse[ws] = lse;
      } else {
        static_cast<TQ*>(p.o)[s.b * p.so.b + (h0 + h) * p.so.h + d] = Elem<TQ>::put(o);
        if (d == 0 && p.lse)
          p.lse[static_cast<long long>(s.b) * p.H + h0 + h] = lse * 0.6931471805599453f;
      }
    }
  }
}

// ------------------------------------------------------------------ the join
// One block per (sequence, query head): outputs of the CTAs that share its
// segment, weighted by their log-sum-exps.  DPAD / 4 threads take a row of
// partial output, the block several rows at once, which are added up in order
// at the end.  Sequences without keys get the empty row (0, -inf).
// (Latency: an empty kernel here costs 1 us, the chain lengths -> CTAs ->
// partial outputs -> sum another 3 to 4; a block per segment, blocks of 64 to
// 512 threads and a join by the last CTA of a segment to finish (counters
// zeroed by a kernel in front) measured the same within 1 us, or slower where
// a segment has many parts.)
constexpr int kJoinThreads = 256;
template <typename T, int DPAD>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams p, int hpb) {
  constexpr int LPR = DPAD / 4, ROWS = kJoinThreads / LPR;  // threads of a row; rows at once
  __shared__ float4 sums[kJoinThreads];
  __shared__ float2 stats[ROWS];  // maximum and weight
  const PagedCache& c = p.c;
  const int b = static_cast<int>(blockIdx.x / p.H), h = static_cast<int>(blockIdx.x % p.H);
  const int hk = h / p.group, hb = (h - hk * p.group) / hpb, hi = (h - hk * p.group) % hpb;
  bool bad = false;
  const int len = clamp_len(c, __ldg(p.lens + b), &bad);
  if (bad && h == 0 && threadIdx.x == 0) atomicOr(c.status, kStatusIndex);
  // This kernel may be placed while the attention kernel runs: from here on
  // that one is complete and its partial states are visible.  (Every block
  // waits, so that this kernel never ends before it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int2 ctas = make_int2(0, -1);
  if (len > 0) ctas = p.ws_cta[(static_cast<long long>(b) * c.Hkv + hk) * p.head_blocks + hb];
  if (ctas.x == ctas.y) return;  // written by that CTA
  const int row = static_cast<int>(threadIdx.x) / LPR, d = 4 * (static_cast<int>(threadIdx.x) % LPR);
  float M = -INFINITY, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto merge = [&](float y, float weight, const float4& x) {
    const float M_new = fmaxf(M, y), mu = M_new == -INFINITY ? 0.f : M_new;
    const float a = exp2f(M - mu), w = exp2f(y - mu);
    M = M_new;
    L = L * a + weight * w;
    acc[0] = fmaf(w, x.x, acc[0] * a), acc[1] = fmaf(w, x.y, acc[1] * a);
    acc[2] = fmaf(w, x.z, acc[2] * a), acc[3] = fmaf(w, x.w, acc[3] * a);
  };
  constexpr int U = 4;  // rows in flight per thread
  for (int cta = ctas.x + row; cta <= ctas.y; cta += U * ROWS) {
    float y[U];
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = cta + u * ROWS;
      y[u] = -INFINITY, x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at <= ctas.y) {
        // the first CTA's piece begins the segment (slot 1), the others' continue it
        const long long r = slot_row(p, at, at == ctas.x ? 1 : 0, hpb, hi);
        if (!JVP_CHECK(at >= 0 && r < 2ll * p.grid * hpb, c.status, kChkGlobalRow)) continue;
        y[u] = p.ws_lse[r];
        // (columns past D of a row are not written: they are not used either)
        x[u] = *reinterpret_cast<const float4*>(p.ws_o + r * DPAD + d);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) merge(y[u], 1.f, x[u]);
  }
  sums[threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  if (d == 0) stats[row] = make_float2(M, L);
  __syncthreads();
  if (row != 0) return;
#pragma unroll
  for (int i = 1; i < ROWS; ++i) merge(stats[i].x, stats[i].y, sums[threadIdx.x + i * LPR]);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  T* dst = static_cast<T*>(p.o) + b * p.so.b + h * p.so.h;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (d + k < c.D) dst[d + k] = Elem<T>::put(acc[k] * inv);
  if (d == 0 && p.lse)
    p.lse[static_cast<long long>(b) * p.H + h] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ launch
template <auto KERN>
cudaError_t launch_with_smem(int bytes, const DecodeParams& p, cudaStream_t stream) {
  const cudaError_t e = allow_shared_memory<KERN>(bytes);
  if (e != cudaSuccess) return e;
  KERN<<<p.grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename TQ, int DPAD, bool E4M3, int NG>
cudaError_t launch_tc(const DecodeParams& p, cudaStream_t stream) {
  constexpr int bytes = 128 + 2 * sizeof(Exchange<DPAD, NG>) + kWarps * Ring<DPAD, E4M3>::WARP;
  static_assert(decode_ctas_per_sm(DPAD, NG, E4M3) * (bytes + 1024) <= 228 * 1024, "resident CTAs");
  return launch_with_smem<decode_tc_kernel<TQ, DPAD, E4M3, NG>>(bytes, p, stream);
}
template <typename TQ, int DPAD, bool E4M3, int HPB>
cudaError_t launch_simt(bool vec, const DecodeParams& p, cudaStream_t stream) {
  constexpr int bytes = sizeof(SimtShared<HPB, DPAD>);
  return vec ? launch_with_smem<decode_simt_kernel<TQ, DPAD, E4M3, HPB, true>>(bytes, p, stream)
             : launch_with_smem<decode_simt_kernel<TQ, DPAD, E4M3, HPB, false>>(bytes, p, stream);
}

template <typename TQ, int DPAD, bool E4M3>
cudaError_t launch_attention(bool tc, bool vec, const DecodeParams& p, cudaStream_t stream) {
  if constexpr (sizeof(TQ) == 2) {
    if (tc)
      return p.group > 8 ? launch_tc<TQ, DPAD, E4M3, 2>(p, stream)
                         : launch_tc<TQ, DPAD, E4M3, 1>(p, stream);
  }
  return p.group == 1 ? launch_simt<TQ, DPAD, E4M3, 1>(vec, p, stream)
                      : launch_simt<TQ, DPAD, E4M3, 4>(vec, p, stream);
}

template <typename TQ>
cudaError_t launch_typed(bool e4m3, bool tc, bool vec, const DecodeParams& p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const bool wide = p.c.D > 64;
  if (p.grid > 0) {
    e = wide ? (e4m3 ? launch_attention<TQ, 128, true>(tc, vec, p, stream)
                     : launch_attention<TQ, 128, false>(tc, vec, p, stream))
             : (e4m3 ? launch_attention<TQ, 64, true>(tc, vec, p, stream)
                     : launch_attention<TQ, 64, false>(tc, vec, p, stream));
    if (e != cudaSuccess || p.direct) return e;
  }
  // The join may be placed on the GPU while the attention kernel still runs
  // (programmatic dependent launch); it waits for it before it reads.
  cudaLaunchConfig_t cfg = {};
  const int hpb = decode_heads_per_block(tc, p.group);
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.c.B) * p.H));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.grid > 0 ? 1 : 0;
  return wide ? cudaLaunchKernelEx(&cfg, decode_join_kernel<TQ, 128>, p, hpb)
              : cudaLaunchKernelEx(&cfg, decode_join_kernel<TQ, 64>, p, hpb);
}

}  // namespace

cudaError_t launch_decode(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
                          cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_typed<float>(e4m3, tc, vec, p, stream);
    case kF16: return launch_typed<__half>(e4m3, tc, vec, p, stream);
    case kBF16: return launch_typed<__nv_bfloat16>(e4m3, tc, vec, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jvp
