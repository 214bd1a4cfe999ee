// rope.cu -- norms of queries and keys per head and rotation by position: on
// dense tensors for training, with tangents and gradients, and on new rows on
// their way into a paged cache.
//
// Per row x (one head of one token, D elements, w the norm's weights):
//   r = (mean x^2 + eps)^(-1/2),  n = r x,  y = R (w n),
// R the rotation of the pairs of the first `rot` columns by the angles of the
// row's position (R^T is R with the sines negated).  With a tangent dx:
//   m = mean(n dx),  dn = r (dx - m n),  dy = R (w dn).
// Backward, for <gy, y> + <gdy, dy>, with a = R^T gy, b = R^T gdy, u = w a, v = w b:
//   gdx = r (v - n mean(v n)),   gw = sum over rows of a n + b dn,
//   gx  = r (u - n mean(u n))
//       + r^2 (n (3 m mean(v n) - mean(v dx)) - dx mean(v n) - m v).
// (dy is bilinear in v and dx, and depends on x through r and n = r x alone.)
// Without norms y = R x, and both directions are one kernel.  All in fp32, one
// rounding per output; the weights' gradients are sums in fp32 of a fixed order.
//
// Bound: memory.  Every row is read once and written once; nothing else is of
// the rows' size.  LANES lanes share a row, each with two 16-byte pieces of it:
// where the two columns of a pair are half a rotation apart, the lane holds both
// columns of its pairs, so the rotation needs no exchange.  A warp takes
// 32 / LANES tokens that follow one another and walks the heads, so the angles
// are loaded once per token and the weights once per side (queries, keys).
//
// A head's rows are fetched again as soon as they are unpacked, so that loads never pause.
//
// Measured, 4 x 4096 tokens, 16 + 4 heads of 128, % of the copy rate: fp32 forward 55 us
// (90 %), with tangents 106 (93 %), gradients 96 (78 %), with tangents 174 (85 %); bf16
// 33 (75 %), 60 (82 %), 57 (65 %) and 130 (57 %): as many instructions and registers for
// half the bytes, which is why elements are taken in pairs.  Rows into the cache, 47k
// tokens, 16/8 heads of 128, 64 columns rotated: 121 us, 94 %; 48 single rows 4.3 us.
// Rows of any layout cost far more, since a warp takes one and reads its columns one by
// one: bf16 heads of 40, or 80 of which 40 are rotated, 205 and 257 us forward, 244 and
// 375 backward, 52k rows into the cache 690 and 790 us (4 to 10 %).
#include <cmath>
#include <type_traits>

#include "debug_checks.cuh"
#include "paged.cuh"
#include "rows.cuh"
#include "sm103_ptx.cuh"

namespace jvp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// ------------------------------------------------------------------ pieces
template <typename T>
struct Piece {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void get(const uint4& w, float (&x)[N]) {
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Rows<T>::get(e[i]);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[N]) {
    uint4 w;
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = Rows<T>::put(x[i]);
    return w;
  }
};

// A lane's two pieces of a row.  Pairs half a rotation apart: lanes below
// `half` (pieces of half the rotated columns) hold pieces l and l + half, the
// others two of the columns behind.  Neighbouring pairs (IL): pieces l and l + LANES.
template <typename T, int LANES, bool IL>
struct Lane {
  static constexpr int N = Piece<T>::N;
  int at[2];  // first columns
  bool on[2], turned[2];
  __device__ __forceinline__ Lane(const RopeParams& p, int l) {
    int piece[2];
    if constexpr (IL) {
      piece[0] = l, piece[1] = l + LANES;
      turned[0] = piece[0] * N < p.rot, turned[1] = piece[1] * N < p.rot;
    } else {
      const int half = p.rot / (2 * N);
      turned[0] = turned[1] = l < half;
      piece[0] = l < half ? l : 2 * l;
      piece[1] = l < half ? l + half : 2 * l + 1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) at[i] = piece[i] * N, on[i] = at[i] < p.D;
  }
};

// The rotation of a pair, and the root of a norm, rounded in one way wherever they
// are compiled: the kernels give the same bits for the same row.
__device__ __forceinline__ void turn_pair(float c, float s, float* a, float* b) {
  const float x = *a, y = *b;
  *a = fmaf(x, c, -__fmul_rn(y, s)), *b = fmaf(y, c, __fmul_rn(x, s));
}
// Elements e, e + 1 as a pair: 16-bit rows are near the issue rate, and the paired
// forms halve the arithmetic (same roundings).
__device__ __forceinline__ float2 two(const float* x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put2(float* x, const float2& y) { x[0] = y.x, x[1] = y.y; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus(const float2& x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float inverse_root(float squares, const RopeParams& p) {
  return rsqrtf(fmaf(squares, p.inv_d, p.eps));
}

template <typename T, int LANES, bool IL>
struct Angles {
  static constexpr int N = Piece<T>::N;
  float c[N], s[N];
  __device__ __forceinline__ void load(const RopeParams& p, const Lane<T, LANES, IL>& lane,
                                       int position, bool on, bool back) {
    const float* row = p.table + static_cast<long long>(position) * p.rot;
    constexpr int W = IL ? N / 2 : N;  // of one piece (or of both)
#pragma unroll
    for (int i = 0; i < (IL ? 2 : 1); ++i) {
      if (!lane.turned[i]) continue;
      if (!on) {  // (zeros: rows of no token add zeros to the weights' gradients)
#pragma unroll
        for (int e = 0; e < W; ++e) c[i * W + e] = s[i * W + e] = 0.f;
        continue;
      }
      const float* at = row + (IL ? lane.at[i] / 2 : lane.at[0]);
#pragma unroll
      for (int e = 0; e < W; e += 2) {  // (columns are even: 8-byte aligned at least)
        const float2 x = __ldg(reinterpret_cast<const float2*>(at + e));
        const float2 y = __ldg(reinterpret_cast<const float2*>(at + p.rot / 2 + e));
        c[i * W + e] = x.x, c[i * W + e + 1] = x.y;
        s[i * W + e] = back ? -y.x : y.x, s[i * W + e + 1] = back ? -y.y : y.y;
      }
    }
  }
  // x = R x, or R^T x with the angles loaded for the way back
  __device__ __forceinline__ void turn(const Lane<T, LANES, IL>& lane, float (&x)[2][N]) const {
    if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!lane.turned[i]) continue;
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          turn_pair(c[(i * N + e) / 2], s[(i * N + e) / 2], &x[i][e], &x[i][e + 1]);
        }
      }
    } else if (lane.turned[0]) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 cc = two(&c[e]), ss = two(&s[e]);
        const float2 a = two(&x[0][e]), b = two(&x[1][e]);
        put2(&x[0][e], fma2(a, cc, minus(mul2(b, ss))));
        put2(&x[1][e], fma2(b, cc, mul2(a, ss)));
      }
    }
  }
};

__device__ __forceinline__ float weight(const RopeParams& p, const void* w, int d) {
  if (p.weight_type == kF32) return __ldg(static_cast<const float*>(w) + d);
  const unsigned short h = __ldg(static_cast<const unsigned short*>(w) + d);
  return p.weight_type == kF16 ? __half2float(__ushort_as_half(h))
                               : __uint_as_float(static_cast<unsigned>(h) << 16);
}
template <typename T, int LANES, bool IL, int N>
__device__ __forceinline__ void load_weights(const RopeParams& p, const void* w,
                                             const Lane<T, LANES, IL>& lane, float (&x)[2][N]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) x[i][e] = lane.on[i] ? weight(p, w, lane.at[i] + e) : 0.f;
}

// Sum over the lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int N>
__device__ __forceinline__ float dot(const float (&a)[2][N], const float (&b)[2][N]) {
  float2 x = both(0.f);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < N; e += 2) x = fma2(two(&a[i][e]), two(&b[i][e]), x);
  return x.x + x.y;
}
// x = f w x
template <int N>
__device__ __forceinline__ void weigh(float (&x)[2][N], const float (&w)[2][N], float f) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < N; e += 2)
      put2(&x[i][e], mul2(mul2(both(f), two(&w[i][e])), two(&x[i][e])));
}
// x = f (x - m n)
template <int N>
__device__ __forceinline__ void project(float (&x)[2][N], const float (&n)[2][N], float m, float f) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < N; e += 2)
      put2(&x[i][e], mul2(both(f), fma2(both(-m), two(&n[i][e]), two(&x[i][e]))));
}

template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, int at, bool on) {
  return on ? __ldg(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0u, 0u, 0u, 0u);
}

// y = R (w n) of a row in place.
template <typename T, int LANES, bool IL, bool NORM, int N>
__device__ __forceinline__ void norm_and_turn(const RopeParams& p, const Lane<T, LANES, IL>& lane,
                                              const Angles<T, LANES, IL>& angles,
                                              const float (&w)[2][N], float (&x)[2][N]) {
  if constexpr (NORM) {
    weigh(x, w, inverse_root(row_sum<LANES>(dot(x, x)), p));
  }
  angles.turn(lane, x);
}

// ------------------------------------------------------------------ dense rows
// Token (of B * N) and its position; false where there is none, or (recorded)
// its position names no row of the table.
__device__ __forceinline__ bool token_of(const RopeDense& d, long long i, int* b, int* n,
                                         int* position) {
  *b = 0, *n = 0, *position = 0;
  if (i >= d.tokens) return false;
  *b = static_cast<int>(i / d.N), *n = static_cast<int>(i - static_cast<long long>(*b) * d.N);
  *position = d.positions ? __ldg(d.positions + *b * d.positions_stride + *n) : *n;
  if (d.r.rot > 0 && (*position < 0 || *position >= d.r.table_rows)) {
    atomicOr(d.r.status, kStatusIndex);
    return false;
  }
  return true;
}

// A warp's work: tokens 32 / LANES at a time, `heads` heads of the list of query
// and key heads.
struct Unit {
  long long token;  // the first of them
  int h0, h1;
};
__device__ __forceinline__ Unit unit_of(const RopeDense& d, long long u, int per) {
  Unit x;
  const long long group = u / d.head_chunks;
  const int chunk = static_cast<int>(u - group * d.head_chunks);
  x.token = group * per;
  x.h0 = chunk * d.heads_per_unit;
  x.h1 = min(x.h0 + d.heads_per_unit, d.H + d.Hkv);
  return x;
}

// TAN: with tangents.  Without norms also the way back.
template <typename T, int LANES, bool IL, bool NORM, bool TAN>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeDense d) {
  constexpr int N = Piece<T>::N, PER = 32 / LANES;
  // heads whose rows are on their way (bf16 33 us with 3, 38 with 2; fp32 55 with 2, 61 with 3;
  // with tangents 60 with 1, 64 with 2)
  constexpr int UN = TAN ? 1 : sizeof(T) == 2 ? 3 : 2;  // heads in flight
  const RopeParams& p = d.r;
  const long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (u >= d.units) return;
  const int l = threadIdx.x & 31;
  const Unit unit = unit_of(d, u, PER);
  const Lane<T, LANES, IL> lane(p, l % LANES);
  int b, n, position;
  const bool on = token_of(d, unit.token + l / LANES, &b, &n, &position);
  Angles<T, LANES, IL> angles;
  angles.load(p, lane, position, on, d.back != 0);
  const bool ons[2] = {on && lane.on[0], on && lane.on[1]};
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int first = side ? d.H : 0;
    const int h0 = max(unit.h0, first), h1 = min(unit.h1, side ? d.H + d.Hkv : d.H);
    if (h0 >= h1) continue;
    float w[2][N];
    if constexpr (NORM) load_weights(p, side ? p.wk : p.wq, lane, w);
    const Strides &si = d.in[side], &st = d.in[2 + side];
    const Strides &so = d.out[side], &sto = d.out[2 + side];
    const T* x_at = static_cast<const T*>(d.x[side]) + b * si.b + n * si.n;
    const T* t_at = static_cast<const T*>(d.x[2 + side]) + (TAN ? b * st.b + n * st.n : 0);
    T* y_at = static_cast<T*>(d.y[side]) + b * so.b + n * so.n;
    T* ty_at = static_cast<T*>(d.y[2 + side]) + (TAN ? b * sto.b + n * sto.n : 0);
    uint4 raw[UN][2], raw_t[UN][2];
    auto fetch = [&](int k, int h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool o = ons[i] && h < h1;
        raw[k][i] = load_piece(x_at + (h - first) * si.h, lane.at[i], o);
        if constexpr (TAN) raw_t[k][i] = load_piece(t_at + (h - first) * st.h, lane.at[i], o);
      }
    };
#pragma unroll
    for (int k = 0; k < UN; ++k) fetch(k, h0 + k);
    for (int h = h0; h < h1; h += UN) {
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        if (h + k >= h1) break;  // uniform over the warp
        float x[2][N], t[2][N];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Piece<T>::get(raw[k][i], x[i]);
          if constexpr (TAN) Piece<T>::get(raw_t[k][i], t[i]);
        }
        fetch(k, h + k + UN);
        if constexpr (NORM) {
          const float r = inverse_root(row_sum<LANES>(dot(x, x)), p);
          if constexpr (TAN) {  // w r (dx - m n), n = r x
            const float m = r * row_sum<LANES>(dot(x, t)) * p.inv_d;
            project(t, x, m * r, 1.f);
            weigh(t, w, r);
          }
          weigh(x, w, r);
        }
        angles.turn(lane, x);
        if constexpr (TAN) angles.turn(lane, t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ons[i] || !JVP_CHECK(lane.at[i] + N <= p.D && n < d.N, p.status, kChkGlobalCol))
            continue;
          *reinterpret_cast<uint4*>(y_at + (h + k - first) * so.h + lane.at[i]) =
              Piece<T>::put(x[i]);
          if constexpr (TAN)
            *reinterpret_cast<uint4*>(ty_at + (h + k - first) * sto.h + lane.at[i]) =
                Piece<T>::put(t[i]);
        }
      }
    }
  }
}

// gx (and gdx) of every row; the block's sums of the weights' gradients go to
// the workspace, [grid][2][D].
//
// Blocks of an SM, and heads whose rows are on their way: bound by latency (ncu: 45 % of
// issue slots, 56 % of DRAM at 4 x 4096 tokens, bf16, loads waited for first), by the
// registers that hold them in turn.  us, 16 + 4 heads of 128: bf16 57 with 4 blocks and 1
// head (2 heads 67, 3 blocks and 2 heads 67), with tangents 130 with 2 blocks and 2 heads
// (heads of 64 33; 3 blocks and 1 head 130, 44); fp32 96 with 4 and 3 (2 heads 99, 3 blocks
// 116), with tangents 174 with 4 and 1 (3 and 2: 194).
template <typename T>
constexpr int bwd_blocks(bool tangents) {
  return tangents && sizeof(T) == 2 ? 2 : 4;
}
template <typename T>
constexpr int bwd_heads(bool tangents) {
  return sizeof(T) == 2 ? (tangents ? 2 : 1) : (tangents ? 1 : 3);
}
template <typename T, int LANES, bool IL, bool TAN>
__global__ void __launch_bounds__(kThreads, bwd_blocks<T>(TAN)) norm_rope_bwd_kernel(const RopeDense d) {
  constexpr int N = Piece<T>::N, PER = 32 / LANES;
  constexpr int UN = bwd_heads<T>(TAN);
  const RopeParams& p = d.r;
  __shared__ float sums[kWarps][LANES][2 * N];
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const Lane<T, LANES, IL> lane(p, l % LANES);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int first = side ? d.H : 0;
    float w[2][N], gw[2][N];
    load_weights(p, side ? p.wk : p.wq, lane, w);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) gw[i][e] = 0.f;
    const Strides &sx = d.in[side], &st = d.in[2 + side], &sg = d.in[4 + side],
                  &sgt = d.in[6 + side];
    const Strides &so = d.out[side], &sto = d.out[2 + side];
#pragma unroll 1
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + warp; u < d.units;
         u += static_cast<long long>(gridDim.x) * kWarps) {
      const Unit unit = unit_of(d, u, PER);
      const int h0 = max(unit.h0, first), h1 = min(unit.h1, side ? d.H + d.Hkv : d.H);
      if (h0 >= h1) continue;
      int b, n, position;
      const bool on = token_of(d, unit.token + l / LANES, &b, &n, &position);
      Angles<T, LANES, IL> angles;
      angles.load(p, lane, position, on, true);
      const bool ons[2] = {on && lane.on[0], on && lane.on[1]};
      const T* x_at = static_cast<const T*>(d.x[side]) + b * sx.b + n * sx.n;
      const T* t_at = static_cast<const T*>(d.x[2 + side]) + (TAN ? b * st.b + n * st.n : 0);
      const T* g_at = static_cast<const T*>(d.x[4 + side]) + b * sg.b + n * sg.n;
      const T* gt_at = static_cast<const T*>(d.x[6 + side]) + (TAN ? b * sgt.b + n * sgt.n : 0);
      T* o_at = static_cast<T*>(d.y[side]) + b * so.b + n * so.n;
      T* ot_at = static_cast<T*>(d.y[2 + side]) + (TAN ? b * sto.b + n * sto.n : 0);
      uint4 rx[UN][2], rg[UN][2], rt[UN][2], rgt[UN][2];
      auto fetch = [&](int k, int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool o = ons[i] && h < h1;
          const int hh = h - first;
          rx[k][i] = load_piece(x_at + hh * sx.h, lane.at[i], o);
          rg[k][i] = load_piece(g_at + hh * sg.h, lane.at[i], o);
          if constexpr (TAN) {
            rt[k][i] = load_piece(t_at + hh * st.h, lane.at[i], o);
            rgt[k][i] = load_piece(gt_at + hh * sgt.h, lane.at[i], o);
          }
        }
      };
#pragma unroll
      for (int k = 0; k < UN; ++k) fetch(k, h0 + k);
      for (int h = h0; h < h1; h += UN) {
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          if (h + k >= h1) break;  // uniform over the warp
          float x[2][N], g[2][N], t[2][N], v[2][N];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            Piece<T>::get(rx[k][i], x[i]), Piece<T>::get(rg[k][i], g[i]);
            if constexpr (TAN) Piece<T>::get(rt[k][i], t[i]), Piece<T>::get(rgt[k][i], v[i]);
          }
          fetch(k, h + k + UN);
          const float root = inverse_root(row_sum<LANES>(dot(x, x)), p);
          const float r = on ? root : 0.f;  // (no token: eps may be 0)
          angles.turn(lane, g);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              const float2 nn = mul2(both(r), two(&x[i][e])), a = two(&g[i][e]);
              put2(&x[i][e], nn);
              put2(&gw[i][e], fma2(a, nn, two(&gw[i][e])));
              put2(&g[i][e], mul2(a, two(&w[i][e])));  // u
            }
          const float un = row_sum<LANES>(dot(g, x)) * p.inv_d;
          if constexpr (TAN) {
            angles.turn(lane, v);
            const float m = row_sum<LANES>(dot(x, t)) * p.inv_d;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                const float2 dn =
                    mul2(both(r), fma2(both(-m), two(&x[i][e]), two(&t[i][e])));
                put2(&gw[i][e], fma2(two(&v[i][e]), dn, two(&gw[i][e])));
                put2(&v[i][e], mul2(two(&v[i][e]), two(&w[i][e])));
              }
            const float vn = row_sum<LANES>(dot(v, x)) * p.inv_d;
            const float vt = row_sum<LANES>(dot(v, t)) * p.inv_d;
            // gx = r (u + of_n n - r (vn dx + m v)), gdx = r (v - vn n)
            const float of_n = r * (3.f * m * vn - vt) - un;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                const float2 y = fma2(both(of_n), two(&x[i][e]), two(&g[i][e]));
                const float2 z = fma2(both(vn), two(&t[i][e]), mul2(both(m), two(&v[i][e])));
                put2(&g[i][e], mul2(both(r), fma2(both(-r), z, y)));
              }
            project(v, x, vn, r);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (ons[i])
                *reinterpret_cast<uint4*>(ot_at + (h + k - first) * sto.h + lane.at[i]) =
                    Piece<T>::put(v[i]);
          } else {
            project(g, x, un, r);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ons[i] && JVP_CHECK(lane.at[i] + N <= p.D && n < d.N, p.status, kChkGlobalCol))
              *reinterpret_cast<uint4*>(o_at + (h + k - first) * so.h + lane.at[i]) =
                  Piece<T>::put(g[i]);
        }
      }
    }
    // over the warp's tokens, then over the warps
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1)
          gw[i][e] += __shfl_xor_sync(0xffffffffu, gw[i][e], o);
        if (l < LANES) sums[warp][l][i * N + e] = gw[i][e];
      }
    __syncthreads();
    if (warp == 0 && l < LANES) {
      float* to = d.ws + (static_cast<long long>(blockIdx.x) * 2 + side) * p.D;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane.on[i])
#pragma unroll
          for (int e = 0; e < N; ++e) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) x += sums[k][l][i * N + e];
            to[lane.at[i] + e] = x;
          }
    }
    __syncthreads();
  }
}

// Weights' gradients from the blocks' sums: a block per side and 8 columns.
constexpr int kJoinCols = 8, kJoinRows = 32;
__global__ void __launch_bounds__(kJoinCols* kJoinRows) norm_rope_join_kernel(const RopeDense d,
                                                                              int blocks) {
  __shared__ float part[kJoinRows][kJoinCols + 1];
  const int col = static_cast<int>(threadIdx.x) % kJoinCols;
  const int row = static_cast<int>(threadIdx.x) / kJoinCols;
  const int c = static_cast<int>(blockIdx.x) * kJoinCols + col, side = static_cast<int>(blockIdx.y);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float x = 0.f;
  if (c < d.r.D)
    for (int k = row; k < blocks; k += kJoinRows)
      x += d.ws[(static_cast<long long>(k) * 2 + side) * d.r.D + c];
  part[row][col] = x;
  __syncthreads();
  if (row != 0 || c >= d.r.D) return;
#pragma unroll
  for (int k = 1; k < kJoinRows; ++k) x += part[k][col];
  (side ? d.gwk : d.gwq)[c] = x;
}

// ------------------------------------------------------------------ any layout
// One row per warp, lane-strided elements (a lane has columns l, l + 32, ...).
constexpr int kSlots = 4;  // D <= 128

struct AnyRow {
  const RopeParams& p;
  int lane, position;
  // f rotated (back: the other way) at column col; f gives any column
  template <typename F>
  __device__ __forceinline__ float turned(const F& f, int col, bool back) const {
    if (col >= p.rot) return f(col);
    const int half = p.rot / 2;
    const int j = p.interleaved ? col >> 1 : (col < half ? col : col - half);
    const bool second = p.interleaved ? (col & 1) : col >= half;
    const int other = p.interleaved ? col ^ 1 : (second ? col - half : col + half);
    const float* row = p.table + static_cast<long long>(position) * p.rot;
    const float c = __ldg(row + j), s = __ldg(row + half + j);
    const float b = __fmul_rn(f(other), s);  // (as turn_pair)
    return fmaf(f(col), c, second != back ? b : -b);
  }
  // sum of f g over the columns
  template <typename F, typename G>
  __device__ __forceinline__ float sum(const F& f, const G& g) const {
    float x = 0.f;
    for (int c = lane; c < p.D; c += 32) x = fmaf(f(c), g(c), x);
    return row_sum<32>(x);
  }
};

template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const RopeDense d) {
  const RopeParams& p = d.r;
  __shared__ float sums[kWarps][32 * kSlots];
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const bool tan = d.x[2] != nullptr || d.x[3] != nullptr, norm = p.wq != nullptr;
  if (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int heads = side ? d.Hkv : d.H;
    const void* w = side ? p.wk : p.wq;
    float gw[kSlots] = {0.f, 0.f, 0.f, 0.f};
    const Strides &sx = d.in[side], &st = d.in[2 + side], &sg = d.in[4 + side],
                  &sgt = d.in[6 + side];
    const Strides &so = d.out[side], &sto = d.out[2 + side];
    const long long rows = d.tokens * heads;
#pragma unroll 1
    for (long long i = static_cast<long long>(blockIdx.x) * kWarps + warp; i < rows;
         i += static_cast<long long>(gridDim.x) * kWarps) {
      const long long token = i / heads;
      const int h = static_cast<int>(i - token * heads);
      int b, n, position;
      if (!token_of(d, token, &b, &n, &position)) continue;  // uniform over the warp
      const AnyRow row{p, l, position};
      auto at = [&](int k, const Strides& s) {
        return static_cast<const T*>(d.x[k + side]) + b * s.b + n * s.n + h * s.h;
      };
      auto value = [](const T* x) { return [x](int c) { return Rows<T>::get(x[c]); }; };
      const auto x = value(at(0, sx));
      const auto t = value(tan ? at(2, st) : nullptr);
      T* y = static_cast<T*>(d.y[side]) + b * so.b + n * so.n + h * so.h;
      T* ty = tan ? static_cast<T*>(d.y[2 + side]) + b * sto.b + n * sto.n + h * sto.h : nullptr;
      const bool back = d.back != 0;
      if (!norm) {
        for (int c = l; c < p.D; c += 32) {
          y[c] = Rows<T>::put(row.turned(x, c, back));
          if (tan) ty[c] = Rows<T>::put(row.turned(t, c, back));
        }
        continue;
      }
      const float r = inverse_root(row.sum(x, x), p);
      const float m = tan ? r * row.sum(x, t) * p.inv_d : 0.f;
      if constexpr (!BWD) {
        const auto u = [&](int c) { return r * weight(p, w, c) * x(c); };
        const auto du = [&](int c) { return r * weight(p, w, c) * (t(c) - m * (r * x(c))); };
        for (int c = l; c < p.D; c += 32) {
          y[c] = Rows<T>::put(row.turned(u, c, false));
          if (tan) ty[c] = Rows<T>::put(row.turned(du, c, false));
        }
      } else {
        const auto g = value(at(4, sg));
        const auto gt = value(tan ? at(6, sgt) : nullptr);
        float a[kSlots], v[kSlots], un = 0.f, vn = 0.f, vt = 0.f;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
          const int c = l + 32 * k;
          a[k] = v[k] = 0.f;
          if (c >= p.D) continue;
          const float nc = r * x(c), wc = weight(p, w, c);
          a[k] = row.turned(g, c, true);
          gw[k] = fmaf(a[k], nc, gw[k]);
          a[k] *= wc;
          un = fmaf(a[k], nc, un);
          if (tan) {
            v[k] = row.turned(gt, c, true);
            gw[k] = fmaf(v[k], r * (t(c) - m * nc), gw[k]);
            v[k] *= wc;
            vn = fmaf(v[k], nc, vn), vt = fmaf(v[k], t(c), vt);
          }
        }
        un = row_sum<32>(un) * p.inv_d;
        if (tan) vn = row_sum<32>(vn) * p.inv_d, vt = row_sum<32>(vt) * p.inv_d;
        const float of_n = r * (3.f * m * vn - vt) - un;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
          const int c = l + 32 * k;
          if (c >= p.D) continue;
          const float nc = r * x(c);
          float gx = fmaf(of_n, nc, a[k]);
          if (tan) {
            gx -= r * (vn * t(c) + m * v[k]);
            ty[c] = Rows<T>::put(r * (v[k] - vn * nc));
          }
          y[c] = Rows<T>::put(r * gx);
        }
      }
    }
    if (BWD) {
#pragma unroll
      for (int k = 0; k < kSlots; ++k) sums[warp][l + 32 * k] = gw[k];
      __syncthreads();
      const int c = static_cast<int>(threadIdx.x);
      if (c < p.D) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) x += sums[k][c];
        d.ws[(static_cast<long long>(blockIdx.x) * 2 + side) * p.D + c] = x;
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ into the cache
// Place and position of packed row r; false where it has none.
__device__ __forceinline__ bool place_of(const AppendParams& a, long long r, int* page, int* row,
                                         int* position) {
  *page = *row = *position = 0;
  if (r >= a.T || !locate_row(a.c, a.cu, a.start, a.T, r, page, row, position)) {
    *page = *row = *position = 0;
    return false;
  }
  if (a.r.rot > 0 && *position >= a.r.table_rows) {
    atomicOr(a.r.status, kStatusIndex);
    *page = *row = *position = 0;
    return false;
  }
  return true;
}
// Rounded to the rows' type first, so that what is cached is what the dense
// kernel and a write of its result would give.
template <typename T, int N>
__device__ __forceinline__ void as_type(float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = Rows<T>::get(Rows<T>::put(x[e]));
}

// Heads: H of queries, then Hkv of keys, then Hkv of values.
template <typename T, int LANES, bool IL, bool NORM, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams a) {
  constexpr int N = Piece<T>::N, PER = 32 / LANES, UN = 4;
  const RopeParams& p = a.r;
  const PagedCache& c = a.c;
  check_sequence_offsets(c, a.cu, a.T, static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x);
  const long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (u >= a.units) return;
  const int l = threadIdx.x & 31;
  const long long group = u / a.head_chunks;
  const int all = a.H + 2 * c.Hkv;
  const int u0 = static_cast<int>(u - group * a.head_chunks) * a.heads_per_unit;
  const int u1 = min(u0 + a.heads_per_unit, all);
  const Lane<T, LANES, IL> lane(p, l % LANES);
  const long long r = group * PER + l / LANES;
  int page, row, position;
  const bool on = place_of(a, r, &page, &row, &position);
  Angles<T, LANES, IL> angles;
  if (u0 < a.H + c.Hkv) angles.load(p, lane, position, on, false);
  const bool ons[2] = {on && lane.on[0], on && lane.on[1]};
#pragma unroll 1
  for (int side = 0; side < 3; ++side) {
    const int first = side == 0 ? 0 : side == 1 ? a.H : a.H + c.Hkv;
    const int h0 = max(u0, first);
    const int h1 = min(u1, side == 0 ? a.H : side == 1 ? a.H + c.Hkv : all);
    if (h0 >= h1) continue;
    float w[2][N];
    if constexpr (NORM)
      if (side < 2) load_weights(p, side ? p.wk : p.wq, lane, w);
    const Strides& si = a.in[side];
    const T* x_at = static_cast<const T*>(a.x[side]) + (on ? r * si.n : 0);
    const Strides& sc = side == 1 ? c.sk : c.sv;
    const long long cached = page * sc.b + row * sc.n;
    for (int h = h0; h < h1; h += UN) {
      uint4 raw[UN][2];
#pragma unroll
      for (int k = 0; k < UN; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[k][i] =  // (not the read-only path: q_out may be q)
              ons[i] && h + k < h1
                  ? *reinterpret_cast<const uint4*>(x_at + (h + k - first) * si.h + lane.at[i])
                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        if (h + k >= h1) break;  // uniform over the warp
        const int hh = h + k - first;
        float x[2][N];
        if (side < 2 || E4M3) {
#pragma unroll
          for (int i = 0; i < 2; ++i) Piece<T>::get(raw[k][i], x[i]);
        }
        if (side < 2) {
          norm_and_turn<T, LANES, IL, NORM>(p, lane, angles, w, x);
#pragma unroll
          for (int i = 0; i < 2; ++i) raw[k][i] = Piece<T>::put(x[i]);
        }
        if (side == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ons[i])
              *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + r * a.sq_out.n +
                                        hh * a.sq_out.h + lane.at[i]) = raw[k][i];
          continue;
        }
        const long long to = cached + hh * sc.h;
        if constexpr (!E4M3) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ons[i] && JVP_CHECK(lane.at[i] + N <= p.D, p.status, kChkGlobalCol))
              *reinterpret_cast<uint4*>(static_cast<T*>(side == 1 ? c.k : c.v) + to + lane.at[i]) =
                  raw[k][i];
        } else {
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            as_type<T>(x[i]);
#pragma unroll
            for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(x[i][e]));
          }
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const unsigned sb = scale_byte(top);
          const float inv = __uint_as_float((254u - sb) << 23);  // 2^-e, e = sb - 127
          uint8_t* const code = static_cast<uint8_t*>(side == 1 ? c.k : c.v) + to;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t y[N / 4];
#pragma unroll
            for (int e = 0; e < N; e += 4)
              y[e / 4] = to_e4m3x2(x[i][e] * inv, x[i][e + 1] * inv) |
                         static_cast<uint32_t>(to_e4m3x2(x[i][e + 2] * inv, x[i][e + 3] * inv)) << 16;
            if (!ons[i] || !JVP_CHECK(lane.at[i] + N <= p.D, p.status, kChkGlobalCol)) continue;
            if constexpr (N == 8)
              *reinterpret_cast<uint2*>(code + lane.at[i]) = make_uint2(y[0], y[1]);
            else
              *reinterpret_cast<uint32_t*>(code + lane.at[i]) = y[0];
          }
          if (on && l % LANES == 0)
            (side == 1 ? c.k_scale : c.v_scale)[(static_cast<long long>(page) * c.Hkv + hh) *
                                                    c.page_size + row] = static_cast<uint8_t>(sb);
        }
      }
    }
  }
}

// Any layout: a warp takes one row of one head.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_append_any_kernel(const AppendParams a) {
  const RopeParams& p = a.r;
  const PagedCache& c = a.c;
  check_sequence_offsets(c, a.cu, a.T, static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x);
  const int l = threadIdx.x & 31;
  const int all = a.H + 2 * c.Hkv;
  const long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long r = u / all;
  if (r >= a.T) return;
  const int hu = static_cast<int>(u - r * all);
  const int side = hu < a.H ? 0 : hu < a.H + c.Hkv ? 1 : 2;
  const int h = hu - (side == 0 ? 0 : side == 1 ? a.H : a.H + c.Hkv);
  int page, row, position;
  if (!place_of(a, r, &page, &row, &position)) return;
  const Strides& si = a.in[side];
  const T* x = static_cast<const T*>(a.x[side]) + r * si.n + h * si.h;
  const void* w = side ? p.wk : p.wq;
  const AnyRow any{p, l, position};
  const bool norm = side < 2 && p.wq != nullptr;
  float rs = 1.f;
  const auto value = [x](int d) { return Rows<T>::get(x[d]); };
  if (norm) rs = inverse_root(any.sum(value, value), p);
  const auto u_of = [&](int d) { return norm ? rs * weight(p, w, d) * value(d) : value(d); };
  T y[kSlots];
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kSlots; ++k) {
    const int d = l + 32 * k;
    if (d >= p.D) continue;
    y[k] = side < 2 ? Rows<T>::put(any.turned(u_of, d, false)) : x[d];
    top = fmaxf(top, fabsf(Rows<T>::get(y[k])));
  }
  __syncwarp();  // q_out may be q, of which lanes read one another's columns
  const Strides& sc = side == 1 ? c.sk : c.sv;
  const long long to = side == 0 ? r * a.sq_out.n + h * a.sq_out.h
                                 : page * sc.b + row * sc.n + h * sc.h;
  if (side == 0 || !E4M3) {
    T* dst = static_cast<T*>(side == 0 ? a.q_out : side == 1 ? c.k : c.v) + to;
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
      if (l + 32 * k < p.D) dst[l + 32 * k] = y[k];
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const unsigned sb = scale_byte(top);
  const float inv = __uint_as_float((254u - sb) << 23);
  uint8_t* dst = static_cast<uint8_t*>(side == 1 ? c.k : c.v) + to;
#pragma unroll
  for (int k = 0; k < kSlots; ++k)
    if (l + 32 * k < p.D)
      dst[l + 32 * k] = static_cast<uint8_t>(to_e4m3x2(Rows<T>::get(y[k]) * inv, 0.f) & 0xFFu);
  if (l == 0)
    (side == 1 ? c.k_scale : c.v_scale)[(static_cast<long long>(page) * c.Hkv + h) * c.page_size +
                                        row] = static_cast<uint8_t>(sb);
}

// ------------------------------------------------------------------ launch
// Lanes of a row: the power of two that covers its pieces, two a lane (4 at least).
template <typename T, typename F>
cudaError_t with_lanes(int D, F&& f) {
  constexpr int N = Piece<T>::N;
  if (D <= 8 * N) return f(std::integral_constant<int, 4>());
  if (D <= 16 * N) return f(std::integral_constant<int, 8>());
  if constexpr (sizeof(T) == 4) return f(std::integral_constant<int, 16>());
  return cudaErrorInvalidValue;
}
template <typename F>
cudaError_t with_bool(bool x, F&& f) {
  return x ? f(std::true_type()) : f(std::false_type());
}
template <typename F>
cudaError_t with_type(DType dt, F&& f) {
  switch (dt) {
    case kF32: return f(float());
    case kF16: return f(__half());
    case kBF16: return f(__nv_bfloat16());
  }
  return cudaErrorInvalidValue;
}

// Units (warps' work) of a group of tokens: its heads in so many parts that `warps` at a
// time take the fewest rounds of heads, a unit's beginning (angles, weights, first loads)
// counted as one and a half.
void split_heads(long long groups, int heads, long long warps, int* per_unit, int* chunks) {
  long long best = -1;
  *per_unit = 1, *chunks = heads > 0 ? heads : 1;
  for (long long c = 1; c <= heads;) {
    const long long n = (heads + c - 1) / c;
    const long long cost = (groups * c + warps - 1) / warps * (2 * n + 3);
    if (best < 0 || cost < best)
      best = cost, *per_unit = static_cast<int>(n), *chunks = static_cast<int>(c);
    if (n == 1) break;
    c = (heads + n - 2) / (n - 1);  // the fewest parts that are smaller
  }
}

cudaError_t launch_join(const RopeDense& d, int blocks, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((d.r.D + kJoinCols - 1) / kJoinCols), 2);
  return launch_dependent(norm_rope_join_kernel, grid, kJoinCols * kJoinRows, 0, stream, d, blocks);
}

}  // namespace

cudaError_t launch_norm_rope(DType dt, bool vec, bool bwd, RopeDense d, int num_sms,
                             cudaStream_t stream) {
  const bool norm = d.r.wq != nullptr, tan = d.x[2] != nullptr || d.x[3] != nullptr;
  // (one at least: without rows the weights' gradients are zeros)
  auto blocks_within = [&](long long blocks, int per_sm) {
    const long long most = static_cast<long long>(num_sms) * per_sm;
    return static_cast<int>(blocks < 1 ? 1 : blocks < most ? blocks : most);
  };
  return with_type(dt, [&](auto t) -> cudaError_t {
    using T = decltype(t);
    if (!vec) {
      const long long rows = d.tokens * (d.H > d.Hkv ? d.H : d.Hkv);
      const long long blocks = (rows + kWarps - 1) / kWarps;
      const int grid = blocks_within(blocks, rope_blocks_per_sm());
      if (bwd && norm) norm_rope_any_kernel<T, true><<<grid, kThreads, 0, stream>>>(d);
      else norm_rope_any_kernel<T, false><<<grid, kThreads, 0, stream>>>(d);
      const cudaError_t e = cudaGetLastError();
      return e != cudaSuccess || !(bwd && norm) ? e : launch_join(d, grid, stream);
    }
    return with_lanes<T>(d.r.D, [&](auto lanes) -> cudaError_t {
      constexpr int LANES = decltype(lanes)::value;
      const long long groups = (d.tokens + 32 / LANES - 1) / (32 / LANES);
      const int per_sm = bwd && norm ? bwd_blocks<T>(tan) : rope_blocks_per_sm();
      split_heads(groups, d.H + d.Hkv, static_cast<long long>(num_sms) * per_sm * kWarps,
                  &d.heads_per_unit, &d.head_chunks);
      d.units = groups * d.head_chunks;
      const long long blocks = (d.units + kWarps - 1) / kWarps;
      return with_bool(d.r.interleaved, [&](auto il) -> cudaError_t {
        return with_bool(tan, [&](auto tg) -> cudaError_t {
          constexpr bool IL = decltype(il)::value, TAN = decltype(tg)::value;
          if (bwd && norm) {
            const int grid = blocks_within(blocks, per_sm);
            norm_rope_bwd_kernel<T, LANES, IL, TAN><<<grid, kThreads, 0, stream>>>(d);
            const cudaError_t e = cudaGetLastError();
            return e != cudaSuccess ? e : launch_join(d, grid, stream);
          }
          if (norm)
            norm_rope_kernel<T, LANES, IL, true, TAN>
                <<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(d);
          else
            norm_rope_kernel<T, LANES, IL, false, TAN>
                <<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(d);
          return cudaGetLastError();
        });
      });
    });
  });
}

cudaError_t launch_cache_append(DType dt, bool e4m3, bool vec, AppendParams a, int num_sms,
                                cudaStream_t stream) {
  const int all = a.H + 2 * a.c.Hkv;
  // a thread for each sequence's offsets
  const long long offsets = a.cu ? (a.c.B + kThreads - 1ll) / kThreads : 0;
  auto grid_for = [&](long long warps) {
    const long long blocks = (warps + kWarps - 1) / kWarps;
    return static_cast<unsigned>(blocks > offsets ? blocks : offsets);
  };
  return with_type(dt, [&](auto t) -> cudaError_t {
    using T = decltype(t);
    return with_bool(e4m3, [&](auto e8) -> cudaError_t {
      constexpr bool E4M3 = decltype(e8)::value;
      if (!vec) {
        cache_append_any_kernel<T, E4M3><<<grid_for(a.T * all), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
      }
      return with_lanes<T>(a.r.D, [&](auto lanes) -> cudaError_t {
        constexpr int LANES = decltype(lanes)::value;
        const long long groups = (a.T + 32 / LANES - 1) / (32 / LANES);
        split_heads(groups, all, static_cast<long long>(num_sms) * rope_blocks_per_sm() * kWarps,
                    &a.heads_per_unit, &a.head_chunks);
        a.units = groups * a.head_chunks;
        return with_bool(a.r.interleaved, [&](auto il) -> cudaError_t {
          return with_bool(a.r.wq != nullptr, [&](auto nm) -> cudaError_t {
            cache_append_kernel<T, LANES, decltype(il)::value, decltype(nm)::value, E4M3>
                <<<grid_for(a.units), kThreads, 0, stream>>>(a);
            return cudaGetLastError();
          });
        });
      });
    });
  });
}

}  // namespace jvp
