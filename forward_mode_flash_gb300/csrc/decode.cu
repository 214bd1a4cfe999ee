// decode.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cached keys and joined.
//
// Per sequence b and query head h, over its n = lens[b] cached keys:
//   s_j = scale q . k_j,  o = sum_j exp(s_j - m) v_j / l,  lse = m + log l,
// with the running maximum m and sum l of an online softmax (fp32).
//
// Bound: memory.  Every cached row is read once by the query heads of its
// group; nothing is reused beyond that, so what counts is bytes in flight: each
// warp keeps its own ring of row groups in shared memory, filled by 16-byte
// asynchronous copies some groups ahead, and no warp waits for another until
// the end of a segment.
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
// is no second kernel.
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
// w_j = 2^(x_j + ev_j - 127 - mw) with its own running maximum mw (x_j the
// logit in log2 units), so no range of scales over- or underflows; the output
// is 2^(mw - m) sum w_j vc_j / l.  Queries become fp16 after a power-of-two
// normalisation per head (their largest magnitude to [2^14, 2^15)), so bf16
// queries of any magnitude keep their 8 bits.
//
// Rounding: the weights are rounded to 16 bits for the matrix product (fp16
// ones with their largest at 2^14, to keep small weights out of the
// subnormals).  With a 16-bit cache the row sum adds the same rounded weights,
// so the output is the exact average under slightly perturbed weights; the
// log-sum-exp uses the unrounded sum.
#include <cmath>

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

// The warps' states of one piece, in shared memory; their accumulators are
// behind it, one row of DPAD + 1 floats per warp and head (bank spread).
template <int HPB, int DPAD>
struct Shared {
  long long scan[kWarps];
  Place place;
  float m[kWarps][HPB], mw[kWarps][HPB], l[kWarps][HPB], lx[kWarps][HPB];
  // factor of each warp's accumulator in the merged output; lse of the piece
  float f[kWarps][HPB], lse[HPB];
  float qs[HPB];  // e4m3: logit factor of a head (scale * log2(e) * 2^eq)
  static constexpr int kAccBytes = kWarps * HPB * (DPAD + 1) * 4;
};
template <int HPB, int DPAD>
constexpr int shared_bytes() {
  return (static_cast<int>(sizeof(Shared<HPB, DPAD>)) + 127) & ~127;
}

struct Segment {
  int b, hk, hb;      // sequence, key/value head, block of its query heads
  int tiles, len;
};

// Walks this CTA's range of the list: calls piece(segment, tile0, tile1, slot)
// for each segment it touches; slot -1: the whole segment is here.
template <int TILE, typename Sh, typename F>
__device__ __forceinline__ void walk(const DecodeParams& p, Sh* sh, F&& piece) {
  const PagedCache& c = p.c;
  const long long HH = static_cast<long long>(c.Hkv) * p.head_blocks;
  bool bad = false;
  if (p.direct) {  // one segment per CTA
    Segment s;
    s.b = static_cast<int>(blockIdx.x / HH);
    const int seg = static_cast<int>(blockIdx.x % HH);
    s.hk = seg / p.head_blocks, s.hb = seg % p.head_blocks;
    s.len = clamp_len(c, __ldg(p.lens + s.b), &bad);
    if (bad && seg == 0 && threadIdx.x == 0) atomicOr(c.status, kStatusIndex);
    s.tiles = tiles_of(s.len, TILE);
    piece(s, 0, s.tiles, -1);
    return;
  }
  const int per = (c.B + kThreads - 1) / kThreads;  // sequences per thread
  const int b_lo = min(c.B, static_cast<int>(threadIdx.x) * per), b_hi = min(c.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(clamp_len(c, __ldg(p.lens + b), &bad), TILE);
  long long seq_total;
  const long long before = block_exclusive<kThreads>(mine, &seq_total, sh->scan);
  const long long W = seq_total * HH;
  const long long G = min(static_cast<long long>(p.grid), W);
  if (static_cast<long long>(blockIdx.x) >= G) return;
  const long long lo = W * blockIdx.x / G, hi = W * (blockIdx.x + 1) / G;
  // the thread whose run of sequences holds tile lo finds the sequence
  if (lo >= before * HH && lo < (before + mine) * HH) {
    long long at = before;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const int t = tiles_of(clamp_len(c, __ldg(p.lens + b), &bad), TILE);
      if (lo < (at + t) * HH) break;
      at += t;
    }
    sh->place.b = b;
    sh->place.before = at;
  }
  __syncthreads();
  int b = sh->place.b;
  long long seq_first = sh->place.before * HH;
  int len = clamp_len(c, __ldg(p.lens + b), &bad), nt = tiles_of(len, TILE);
  for (long long at = lo; at < hi;) {
    while (at >= seq_first + nt * HH) {  // next sequence with keys (at < hi <= W: there is one)
      seq_first += nt * HH;
      ++b;
      len = clamp_len(c, __ldg(p.lens + b), &bad), nt = tiles_of(len, TILE);
    }
    const int seg = static_cast<int>((at - seq_first) / nt);
    Segment s;
    s.b = b, s.hk = seg / p.head_blocks, s.hb = seg % p.head_blocks;
    s.tiles = nt, s.len = len;
    const long long first = seq_first + static_cast<long long>(seg) * nt;
    const int t0 = static_cast<int>(at - first);
    const int t1 = static_cast<int>(min(hi - first, static_cast<long long>(nt)));
    const int slot = (t0 == 0 && t1 == nt) ? -1 : (t0 > 0 ? 0 : 1);
    piece(s, t0, t1, slot);
    at = first + t1;
  }
}

// Merged output of a piece: from the warps' states in shared memory to the
// output tensor (slot < 0) or the workspace.
template <typename T, int HPB, int DPAD>
__device__ __forceinline__ void store_piece(const DecodeParams& p, Shared<HPB, DPAD>* sh,
                                            const float* acc, const Segment& s, int slot) {
  const int D = p.c.D;
  const int h0 = s.hk * p.group + s.hb * HPB;            // first query head
  const int nh = min(HPB, p.group - s.hb * HPB);         // heads of this block
  for (int e = threadIdx.x; e < nh * DPAD; e += kThreads) {
    const int h = e / DPAD, d = e % DPAD;
    if (d >= D) continue;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) o += sh->f[w][h] * acc[(w * HPB + h) * (DPAD + 1) + d];
    if (slot < 0) {
      T* dst = static_cast<T*>(p.o) + s.b * p.so.b + (h0 + h) * p.so.h + d;
      *dst = Elem<T>::put(o);
    } else {
      p.ws_o[((static_cast<long long>(blockIdx.x) * 2 + slot) * HPB + h) * D + d] = o;
    }
  }
  if (threadIdx.x < nh) {
    const int h = threadIdx.x;
    if (slot < 0) {
      if (p.lse)
        p.lse[static_cast<long long>(s.b) * p.H + h0 + h] = sh->lse[h] * 0.6931471805599453f;
    } else {
      p.ws_lse[(static_cast<long long>(blockIdx.x) * 2 + slot) * HPB + h] = sh->lse[h];
    }
  }
}

// Factors of the warps' accumulators, from their (m, mw, l, lx): the output is
// sum_w f_w acc_w with f_w = 2^(base_w - M) / sum_w 2^(m_w - M) l_w, base_w the
// exponent that acc_w is relative to (less `shift`), and the log-sum-exp (log2
// units) of the piece.  One thread per head.
template <int HPB, int DPAD>
__device__ __forceinline__ void merge_stats(Shared<HPB, DPAD>* sh, float shift) {
  if (threadIdx.x < HPB) {
    const int h = threadIdx.x;
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh->m[w][h]);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f, lx = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float a = exp2f(sh->m[w][h] - mu);
      l += a * sh->l[w][h];
      lx += a * sh->lx[w][h];
    }
    // (l may be NaN: a NaN among the logits reaches every output of the row)
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int w = 0; w < kWarps; ++w) {
      const float base = sh->mw[w][h];
      sh->f[w][h] = base == -INFINITY ? 0.f : exp2f(base - shift - mu) * inv;
    }
    sh->lse[h] = lx == 0.f ? -INFINITY : mu + log2f(lx);
  }
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

// The ring of one warp: kDecodeStages groups of KT keys, K rows then V rows.
template <int DPAD, bool E4M3>
struct Ring {
  static constexpr int ROWB = DPAD * (E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int KT = decode_warp_keys(DPAD, E4M3);
  static constexpr int PIECES = ROWB / 16;
  static constexpr int STAGE = 2 * KT * ROWB;
  static constexpr int WARP = kDecodeStages * STAGE;
  // byte offset of 16-byte piece x of a row
  static __device__ __forceinline__ int k_at(int row, int x) {
    return row * ROWB + ((PIECES >= 8 ? x ^ ((row & 1) << 2) : x) << 4);
  }
  static __device__ __forceinline__ int v_at(int row, int x) {
    return KT * ROWB + row * ROWB + ((PIECES >= 8 ? x ^ (row & 6) : x ^ ((row >> 1) & 3)) << 4);
  }
};

// TQ: type of q and o, and of a 16-bit cache.  NG: groups of 8 query heads.
template <typename TQ, int DPAD, bool E4M3, int NG>
__global__ void __launch_bounds__(kThreads, decode_ctas_per_sm(DPAD, NG))
    decode_tc_kernel(const DecodeParams p) {
  using R = Ring<DPAD, E4M3>;
  constexpr int HPB = 8 * NG;
  constexpr int KT = R::KT, RG = KT / 16, TILE = kWarps * KT, ST = kDecodeStages;
  static_assert(ST == 2, "one group is read while the next is copied");
  constexpr bool kBF16 = Elem<TQ>::kBF16 && !E4M3;  // operand type of the products
  constexpr float kShift = kBF16 ? 0.f : 14.f;      // fp16 weights: largest at 2^14
  constexpr int KS = DPAD / 16;                     // contraction steps of S^T
  constexpr int EPC = E4M3 ? 16 : 8;                // elements of a 16-byte piece
  constexpr int KSP = EPC / 4;                      // contraction steps per K piece
  constexpr int KP = DPAD / (4 * EPC);              // K pieces per lane and key
  constexpr int MT = DPAD / 16;                     // 16-column tiles of O^T
  constexpr int VW = E4M3 ? DPAD / 32 : 4;          // 32-bit words of a V piece (8 lanes a row)
  constexpr int VP = E4M3 ? 1 : DPAD / 64;          // V pieces per lane and key
  constexpr int VE = E4M3 ? DPAD / 8 : 8;           // elements of a V piece
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto* sh = reinterpret_cast<Shared<HPB, DPAD>*>(smem_raw);
  // the rings; at the end of a piece the accumulators lie over them
  uint8_t* rings = smem_raw + shared_bytes<HPB, DPAD>();
  float* acc_sh = reinterpret_cast<float*>(rings);
  const PagedCache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(rings) + warp * R::WARP;
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
  walk<TILE>(p, sh, [&](const Segment& s, int t0, int t1, int slot) {
    const int h0 = s.hk * p.group + s.hb * HPB;
    const int nh = min(HPB, p.group - s.hb * HPB);
    __syncthreads();  // the previous piece's use of shared memory is over

    auto first_key = [&](int it) { return (t0 + it) * TILE + warp * KT; };
    const int n_it = t1 - t0;
    // Block-table entry of this lane's key of group it (its 16-key run's first
    // key where runs lie in one page), unchecked, and that key's row of the
    // page.  Loaded a group ahead of the copies that need it.
    int raw = -1, row = 0;
    bool looked = false;
    auto look_up = [&](int it) {
      const int j = first_key(it) + (runs ? (KT == 32 ? lane & 16 : 0) : lane);
      looked = it < n_it && (runs || lane < KT) && j < s.len;
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
    uint32_t keep_next = 0;
    auto issue = [&](int it) {
      const int j0 = first_key(it);
      if (it < n_it && j0 < s.len) {
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
            copy_async16(dst + R::k_at(r, x), kr + xcol, on);
            copy_async16(dst + R::v_at(r, x), vr + xcol, on);
          }
        }
      }
      copy_async_commit();
    };
    look_up(0);
    issue(0);
    look_up(1);

    // ---- Q^T operand: lane (g, t) holds head g (+ 8 n), permuted to match K
    uint32_t qf[NG][KS][2];
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
        if (warp == 0 && t == 0)
          sh->qs[h] = p.scale_log2 * __uint_as_float(static_cast<unsigned>(127 + ec) << 23);
      }
    }
    if constexpr (E4M3) __syncthreads();
    float qs[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) qs[n][i] = E4M3 ? sh->qs[n * 8 + 2 * t + i] : p.scale_log2;

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

    for (int it = 0; it < n_it && first_key(it) < s.len; ++it) {
      copy_async_wait<0>();
      __syncwarp();  // every lane's copies of group it are in; group it - 1 has been read
      const unsigned sb = sb_next;
      const uint32_t keep = keep_next;
      issue(it + 1);
      look_up(it + 2);
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
#pragma unroll
        for (int r = 0; r < 2 * RG; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = sc[r / 2][n][2 * (r & 1) + i] * (E4M3 ? kscale[r] * qs[n][i] : qs[n][i]);
            x[r][i] = kept(g + 8 * r) ? y : -INFINITY;
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = -INFINITY, topw = -INFINITY;
#pragma unroll
          for (int r = 0; r < 2 * RG; ++r) {
            top = fmaxf(top, x[r][i]);
            if constexpr (E4M3) topw = fmaxf(topw, x[r][i] + vexp[r]);
          }
          const float m_new = fmaxf(m[n][i], max_over_g(top));
          const float mu = m_new == -INFINITY ? 0.f : m_new;
          const float a_m = exp2f(m[n][i] - mu);
          l[n][i] *= a_m, lx[n][i] *= a_m;
          float a_w = a_m, mwu = mu;
          if constexpr (E4M3) {
            const float mw_new = fmaxf(mw[n][i], max_over_g(topw));
            mwu = mw_new == -INFINITY ? 0.f : mw_new;
            a_w = exp2f(mw[n][i] - mwu);
            mw[n][i] = mw_new;
          } else {
            mw[n][i] = m_new;
          }
          m[n][i] = m_new;
#pragma unroll
          for (int r = 0; r < 2 * RG; ++r) {
            if constexpr (E4M3) {
              const float e = ex2_approx(x[r][i] - mu);
              l[n][i] += e, lx[n][i] += e;
              pw[r][i] = ex2_approx(x[r][i] + vexp[r] - mwu + kShift);
            } else {
              pw[r][i] = ex2_approx(x[r][i] - mwu + kShift);
            }
          }
          if (__any_sync(0xffffffffu, a_w != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[n][mt][i] *= a_w;
              acc[n][mt][2 + i] *= a_w;
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

    // ---- join of the four warps
    copy_async_wait<0>();
    __syncthreads();  // no ring is read any more
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ls = sum_over_g(l[n][i]), lxs = sum_over_g(lx[n][i]);
        if (g == 0) {
          const int h = n * 8 + 2 * t + i;
          sh->m[warp][h] = m[n][i];
          sh->mw[warp][h] = mw[n][i];
          // 16-bit caches sum the weights as shifted for the product
          sh->l[warp][h] = E4M3 ? ls : ls * exp2f(-kShift);
          sh->lx[warp][h] = E4M3 ? lxs : lxs * exp2f(-kShift);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int d = E4M3 ? g * VE + 2 * mt : (g + 8 * (mt / 4)) * 8 + 2 * (mt % 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc_sh[(warp * HPB + n * 8 + 2 * t + (i & 1)) * (DPAD + 1) + d + (i >> 1)] = acc[n][mt][i];
      }
    }
    __syncthreads();
    merge_stats(sh, kShift);
    __syncthreads();
    store_piece<TQ, HPB, DPAD>(p, sh, acc_sh, s, slot);
  });
}

// ------------------------------------------------------------------ CUDA cores
// Any type and alignment: fp32 arithmetic.  Four lanes share a key (lane t
// takes the columns 4 (t + 4 i) .. + 3), a warp's 16 keys go in two rounds of
// eight, and a CTA takes HPB query heads, each lane summing its own keys'
// weighted values until the end of the piece.
template <typename T, bool VEC>
__device__ __forceinline__ float4 load4(const T* row, int d, int D) {
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (VEC) {
    if (d < D) {
      if constexpr (sizeof(T) == 4) {
        f = __ldg(reinterpret_cast<const float4*>(row + d));
      } else if constexpr (sizeof(T) == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + d));
        const float2 a = unpack2(w.x, Elem<T>::kBF16), b = unpack2(w.y, Elem<T>::kBF16);
        f = make_float4(a.x, a.y, b.x, b.y);
      } else {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + d));
        const uint32_t a = e4m3x2_to_half2(w & 0xFFFFu), b = e4m3x2_to_half2(w >> 16);
        const float2 fa = unpack2(a, false), fb = unpack2(b, false);
        f = make_float4(fa.x, fa.y, fb.x, fb.y);
      }
    }
  } else {
    float* e = &f.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < D) {
        if constexpr (sizeof(T) == 1) e[i] = unpack2(e4m3x2_to_half2(row[d + i]), false).x;
        else e[i] = Elem<T>::get(row[d + i]);
      }
  }
  return f;
}

template <typename TQ, int DPAD, bool E4M3, int HPB, bool VEC>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(const DecodeParams p) {
  constexpr int NC = DPAD / 16;  // 4-column pieces per lane
  constexpr int TILE = kDecodeSimtTile, KT = TILE / kWarps;
  static_assert(KT == 16, "a warp takes two rounds of eight keys");
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto* sh = reinterpret_cast<Shared<HPB, DPAD>*>(smem_raw);
  auto* sq = reinterpret_cast<float(*)[DPAD]>(smem_raw + shared_bytes<HPB, DPAD>());
  float* acc_sh = reinterpret_cast<float*>(sq + HPB);
  const PagedCache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int D = c.D;
  using TC = typename std::conditional<E4M3, uint8_t, TQ>::type;
  const TC* kc = static_cast<const TC*>(c.k);
  const TC* vc = static_cast<const TC*>(c.v);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  walk<TILE>(p, sh, [&](const Segment& s, int t0, int t1, int slot) {
    const int h0 = s.hk * p.group + s.hb * HPB;
    const int nh = min(HPB, p.group - s.hb * HPB);
    __syncthreads();
    for (int e = threadIdx.x; e < HPB * DPAD; e += kThreads) {
      const int h = e / DPAD, d = e % DPAD;
      sq[h][d] = (h < nh && d < D)
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
    for (int tile = t0; tile < t1; ++tile) {
      const int j0 = tile * TILE + warp * KT;
      if (j0 >= s.len) break;
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {
        const int j = j0 + 8 * r + g;
        bool on = j < s.len;
        long long ko = 0, vo = 0, so = 0;
        if (on) {
          int entry, row;
          split_position(c, j, &entry, &row);
          const int page = page_of(c, s.b, entry);
          on = page >= 0;
          if (on) {
            ko = page * c.sk.b + s.hk * c.sk.h + row * c.sk.n;
            vo = page * c.sv.b + s.hk * c.sv.h + row * c.sv.n;
            so = (static_cast<long long>(page) * c.Hkv + s.hk) * c.page_size + row;
          }
        }
        float4 x[NC];
#pragma unroll
        for (int u = 0; u < NC; ++u)
          x[u] = on ? load4<TC, VEC>(kc + ko, 4 * (t + 4 * u), D) : make_float4(0.f, 0.f, 0.f, 0.f);
        float ks = p.scale_log2, vs = 1.f;
        if (E4M3 && on) {
          ks *= scale_value(__ldg(c.k_scale + so));
          vs = scale_value(__ldg(c.v_scale + so));
        }
        float w[HPB];
#pragma unroll
        for (int h = 0; h < HPB; ++h) {
          float dot = 0.f;
#pragma unroll
          for (int u = 0; u < NC; ++u) {
            const float4 q = *reinterpret_cast<const float4*>(&sq[h][4 * (t + 4 * u)]);
            dot = fmaf(x[u].x, q.x, fmaf(x[u].y, q.y, fmaf(x[u].z, q.z, fmaf(x[u].w, q.w, dot))));
          }
          dot += __shfl_xor_sync(0xffffffffu, dot, 1);
          dot += __shfl_xor_sync(0xffffffffu, dot, 2);
          w[h] = on ? dot * ks : -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < NC; ++u)
          x[u] = on ? load4<TC, VEC>(vc + vo, 4 * (t + 4 * u), D) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < HPB; ++h) {
          const float m_new = fmaxf(m[h], max_over_g(w[h]));
          const float mu = m_new == -INFINITY ? 0.f : m_new;
          const float a = exp2f(m[h] - mu);
          const float e = exp2f(w[h] - mu);
          m[h] = m_new;
          l[h] = l[h] * a + e;
          const float ev = e * vs;
#pragma unroll
          for (int u = 0; u < NC; ++u) {
            acc[h][u].x = fmaf(ev, x[u].x, acc[h][u].x * a);
            acc[h][u].y = fmaf(ev, x[u].y, acc[h][u].y * a);
            acc[h][u].z = fmaf(ev, x[u].z, acc[h][u].z * a);
            acc[h][u].w = fmaf(ev, x[u].w, acc[h][u].w * a);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < HPB; ++h) {
      const float ls = sum_over_g(l[h]);
      if (lane == 0) sh->m[warp][h] = sh->mw[warp][h] = m[h], sh->l[warp][h] = sh->lx[warp][h] = ls;
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const float4 a = make_float4(sum_over_g(acc[h][u].x), sum_over_g(acc[h][u].y),
                                     sum_over_g(acc[h][u].z), sum_over_g(acc[h][u].w));
        if (g == 0) {
          float* dst = acc_sh + (warp * HPB + h) * (DPAD + 1) + 4 * (t + 4 * u);
          dst[0] = a.x, dst[1] = a.y, dst[2] = a.z, dst[3] = a.w;
        }
      }
    }
    __syncthreads();
    merge_stats(sh, 0.f);
    __syncthreads();
    store_piece<TQ, HPB, DPAD>(p, sh, acc_sh, s, slot);
  });
}

// ------------------------------------------------------------------ the join
// One warp per (sequence, query head): outputs of the CTAs that share its
// segment, weighted by their log-sum-exps, in CTA order.  Sequences without
// keys get the empty row (0, -inf).
template <typename T>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const DecodeParams p, int hpb,
                                                               int tile) {
  const PagedCache& c = p.c;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int b = static_cast<int>(item / p.H), h = static_cast<int>(item % p.H);
  bool bad = false;
  long long before = 0, total = 0;
  for (int i = lane; i < c.B; i += 32) {
    const int nt = tiles_of(clamp_len(c, __ldg(p.lens + i), &bad), tile);
    total += nt;
    if (i < b) before += nt;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (bad && item == 0) atomicOr(c.status, kStatusIndex);
  // This kernel may be placed while the attention kernel runs: from here on
  // that one is complete and its partial states are visible.  (Every warp
  // waits, so that this kernel never ends before it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b >= c.B) return;
  T* dst = static_cast<T*>(p.o) + b * p.so.b + h * p.so.h;
  const int nt = tiles_of(clamp_len(c, __ldg(p.lens + b), &bad), tile);
  if (nt == 0) {
    for (int d = lane; d < c.D; d += 32) dst[d] = Elem<T>::put(0.f);
    if (lane == 0 && p.lse) p.lse[static_cast<long long>(b) * p.H + h] = -INFINITY;
    return;
  }
  const long long HH = static_cast<long long>(c.Hkv) * p.head_blocks;
  const long long W = total * HH, G = min(static_cast<long long>(p.grid), W);
  const int hk = h / p.group, hb = (h - hk * p.group) / hpb, hi = (h - hk * p.group) % hpb;
  const long long first = before * HH + static_cast<long long>(hk * p.head_blocks + hb) * nt;
  // CTA c holds tiles [W c / G, W (c + 1) / G): the one that holds tile x
  const long long c0 = ((first + 1) * G - 1) / W, c1 = ((first + nt) * G - 1) / W;
  if (c0 == c1) return;  // written by that CTA
  // the first CTA's piece begins the segment (slot 1), the others' continue it
  auto slot = [&](long long cta) { return (cta * 2 + (cta == c0 ? 1 : 0)) * hpb + hi; };
  float M = -INFINITY;
  for (long long cta = c0 + lane; cta <= c1; cta += 32) M = fmaxf(M, p.ws_lse[slot(cta)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long base = c0; base <= c1; base += 32) {
    const long long cta = base + lane;
    const float w = cta <= c1 ? exp2f(p.ws_lse[slot(cta)] - mu) : 0.f;
    const int n = static_cast<int>(min(32ll, c1 - base + 1));
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.ws_o + slot(base + i) * c.D;
      L += wi;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (lane + 32 * u < c.D) acc[u] = fmaf(wi, src[lane + 32 * u], acc[u]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (lane + 32 * u < c.D) dst[lane + 32 * u] = Elem<T>::put(acc[u] * inv);
  if (lane == 0 && p.lse)
    p.lse[static_cast<long long>(b) * p.H + h] =
        L == 0.f ? -INFINITY : (mu + log2f(L)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ launch
template <typename K>
cudaError_t launch_with_smem(K kern, int bytes, const DecodeParams& p, cudaStream_t stream) {
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  kern<<<p.grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename TQ, int DPAD, bool E4M3, int NG>
cudaError_t launch_tc(const DecodeParams& p, cudaStream_t stream) {
  using S = Shared<8 * NG, DPAD>;
  constexpr int rings = kWarps * Ring<DPAD, E4M3>::WARP;
  constexpr int bytes =
      shared_bytes<8 * NG, DPAD>() + (rings > S::kAccBytes ? rings : S::kAccBytes);
  static_assert(decode_ctas_per_sm(DPAD, NG) * (bytes + 1024) <= 228 * 1024, "resident CTAs");
  return launch_with_smem(decode_tc_kernel<TQ, DPAD, E4M3, NG>, bytes, p, stream);
}
template <typename TQ, int DPAD, bool E4M3>
cudaError_t launch_simt(bool vec, const DecodeParams& p, cudaStream_t stream) {
  constexpr int HPB = DPAD > 64 ? 2 : 4;
  constexpr int bytes =
      shared_bytes<HPB, DPAD>() + HPB * DPAD * 4 + Shared<HPB, DPAD>::kAccBytes;
  return vec ? launch_with_smem(decode_simt_kernel<TQ, DPAD, E4M3, HPB, true>, bytes, p, stream)
             : launch_with_smem(decode_simt_kernel<TQ, DPAD, E4M3, HPB, false>, bytes, p, stream);
}

template <typename TQ, int DPAD, bool E4M3>
cudaError_t launch_attention(bool tc, bool vec, const DecodeParams& p, cudaStream_t stream) {
  if constexpr (sizeof(TQ) == 2) {
    if (tc)
      return p.group > 8 ? launch_tc<TQ, DPAD, E4M3, 2>(p, stream)
                         : launch_tc<TQ, DPAD, E4M3, 1>(p, stream);
  }
  return launch_simt<TQ, DPAD, E4M3>(vec, p, stream);
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
  const long long rows = static_cast<long long>(p.c.B) * p.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.grid > 0 ? 1 : 0;
  const int tile = decode_tile(tc, p.c.D, e4m3);
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<TQ>, p,
                            decode_heads_per_block(tc, p.c.D, p.group), tile);
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
