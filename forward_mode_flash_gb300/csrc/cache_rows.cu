// cache_rows.cu -- rows of keys and values into and out of a paged cache.
//
// Writing in 8 bits: for each (row, head), with top = max |x| over the head
// dimension, the scale is the smallest power of two 2^e, e in [-127, 120],
// with top <= 448 * 2^e, and a code is x / 2^e rounded to the nearest e4m3
// value (ties to even).  e follows from the bits of top: with top = f * 2^k,
// 1 <= f < 2, it is k - 8 where f <= 1.75 (448 = 1.75 * 2^8) and k - 7 above.
// Dividing by a power of two is exact, so the code is the one rounding of the
// definition, whatever the input type.  A NaN is kept as e4m3's NaN and does
// not count for top; an infinity gives e = 120 and reads back as infinity.
//
// Both directions are bound by memory: a row is read once and written once.
// One warp takes one row (all heads of K and V), so its place in the cache
// (a binary search in cu_seqlens and one block-table entry) is looked up once;
// a group of lanes takes one head of K or V with 16 bytes per lane and access
// of the 16- or 32-bit side, several heads at once so that their loads are in
// flight together.  Writing e4m3 is near the issue rate too: the largest
// magnitude of 16-bit rows is found on packed pairs (79 -> 67 us in the case
// below) and a lane takes two pieces of a row where they fit (67 -> 56 us).
// Measured in a CUDA graph, 56.8k rows of 12 sequences, 8 heads of 128: bf16 to
// and from e4m3 57 us written and 60 us read, 91 and 86 % of the copy rate over
// 350 MB; bf16 as it is 71 and 71 us, 96 %; fp32 138 and 138 us, 99 %.  Rows off
// their 16-byte alignment take the kernels for any layout, one head after the
// other: bf16 as it is 184 and 158 us (37 and 43 %).
#include <cmath>
#include <type_traits>

#include "debug_checks.cuh"
#include "paged.cuh"

namespace jvp {
namespace {

constexpr int kWarps = 4;  // rows per block

template <typename T>
struct Rows;  // conversions of a row's element type
template <>
struct Rows<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Rows<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Rows<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// Looks at the offsets of one sequence per thread of the grid (which has as many).
__device__ __forceinline__ void check_offsets(const CacheRowsParams& p) {
  const long long i = static_cast<long long>(blockIdx.x) * (kWarps * 32) + threadIdx.x;
  if (!p.cu || i >= p.c.B) return;
  const int r0 = __ldg(p.cu + i), r1 = __ldg(p.cu + i + 1);
  if (r0 < 0 || r1 < r0 || r1 > p.T) atomicOr(p.c.status, kStatusIndex);
}

// Where row r of the packed tensors lives in the cache: false if it belongs to
// no sequence, or (recorded in the status word) its sequence's offsets or its
// place are out of range.
__device__ __forceinline__ bool locate(const CacheRowsParams& p, long long r, int* page, int* row) {
  int b;
  long long first;
  if (p.cu) {
    // last b with cu[b] <= r
    int lo = -1, hi = p.c.B;  // cu[lo] <= r < cu[hi], the ends taken as given
    while (hi - lo > 1) {
      const int mid = lo + ((hi - lo) >> 1);  // (lo + hi may pass 2^31)
      if (__ldg(p.cu + mid) <= r) lo = mid;
      else hi = mid;
    }
    // rows before the first sequence and behind the last are in none
    if (lo < 0) return false;
    b = lo;
    first = __ldg(p.cu + b);
    const int end = __ldg(p.cu + b + 1);
    if (end <= r || first < 0 || end > p.T) return false;  // (check_offsets records what is wrong)
  } else {
    b = static_cast<int>(r);
    first = r;
  }
  const long long pos = (p.start ? static_cast<long long>(__ldg(p.start + b)) : 0ll) + (r - first);
  const long long most = static_cast<long long>(p.c.max_pages) * p.c.page_size;
  if (pos < 0 || pos >= most) {
    atomicOr(p.c.status, kStatusIndex);
    return false;
  }
  int entry;
  split_position(p.c, static_cast<int>(pos), &entry, row);
  *page = page_of(p.c, b, entry);
  return *page >= 0;
}

// Biased exponent (the scale byte) for a row whose largest magnitude is top.
__device__ __forceinline__ unsigned scale_byte(float top) {
  const unsigned bits = __float_as_uint(top);
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 0 ? 0u : static_cast<unsigned>(e);
}

__device__ __forceinline__ uint16_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Largest magnitude of a group of LANES lanes' PC 16-byte pieces of a row (NaN
// not counted).
template <int LANES, int PC>
__device__ __forceinline__ float group_top(const float*, const uint4 (&x)[PC]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < PC; ++i)
    top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(x[i].x)), fabsf(__uint_as_float(x[i].y))),
                           fmaxf(fabsf(__uint_as_float(x[i].z)), fabsf(__uint_as_float(x[i].w)))));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}
template <typename T2>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  const T2 m = __hmax2(*reinterpret_cast<const T2*>(&a), *reinterpret_cast<const T2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T2, int LANES, int PC>
__device__ __forceinline__ uint32_t packed_top(const uint4 (&x)[PC]) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < PC; ++i) {
    m = pair_max<T2>(pair_max<T2>(m, x[i].x & kAbs), x[i].y & kAbs);
    m = pair_max<T2>(m, pair_max<T2>(x[i].z & kAbs, x[i].w & kAbs));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    m = pair_max<T2>(m, __shfl_xor_sync(0xffffffffu, m, o));
  return pair_max<T2>(m, m >> 16);  // low half
}
template <int LANES, int PC>
__device__ __forceinline__ float group_top(const __half*, const uint4 (&x)[PC]) {
  const uint32_t m = packed_top<__half2, LANES>(x);
  return __low2float(*reinterpret_cast<const __half2*>(&m));
}
template <int LANES, int PC>
__device__ __forceinline__ float group_top(const __nv_bfloat16*, const uint4 (&x)[PC]) {
  return __uint_as_float(packed_top<__nv_bfloat162, LANES>(x) << 16);
}

// Codes of 16 bytes of a row (4 or 8 of them).
template <typename T>
__device__ __forceinline__ void encode(const uint4& x, float inv, uint32_t (&c)[4 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); i += 4)
    c[i / 4] = to_e4m3x2(Rows<T>::get(e[i]) * inv, Rows<T>::get(e[i + 1]) * inv) |
               (static_cast<uint32_t>(to_e4m3x2(Rows<T>::get(e[i + 2]) * inv,
                                                Rows<T>::get(e[i + 3]) * inv))
                << 16);
}
// 16 bytes of a row from their codes.
template <typename T>
__device__ __forceinline__ uint4 decode(const uint32_t (&c)[4 / sizeof(T)], float s) {
  constexpr int VEC = 16 / sizeof(T);
  uint4 x;
  T* e = reinterpret_cast<T*>(&x);
#pragma unroll
  for (int i = 0; i < VEC; i += 4) {
    uint32_t h2[2];
    e4m3x4_to_half2x2(c[i / 4], h2[0], h2[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[k]));
      e[i + 2 * k] = Rows<T>::put(f.x * s);
      e[i + 2 * k + 1] = Rows<T>::put(f.y * s);
    }
  }
  return x;
}
// W 32-bit words of codes at a time, as one access.
template <int W>
__device__ __forceinline__ void put_words(uint8_t* dst, const uint32_t (&c)[W]) {
  if constexpr (W == 1) *reinterpret_cast<uint32_t*>(dst) = c[0];
  else if constexpr (W == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
}
template <int W>
__device__ __forceinline__ void get_words(const uint8_t* src, uint32_t (&c)[W]) {
  if constexpr (W == 1) {
    c[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (W == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
    c[0] = x.x, c[1] = x.y;
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
    c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
  }
}

// What a lane group works on: rows of K heads 0 .. Hkv - 1, then of V heads.
struct HeadRow {
  int h;
  bool v, on;
};
__device__ __forceinline__ HeadRow head_row(const PagedCache& c, int i, bool in_row) {
  HeadRow r;
  r.v = i >= c.Hkv;
  r.h = r.v ? i - c.Hkv : i;
  r.on = i < 2 * c.Hkv && in_row;
  return r;
}

// ------------------------------------------------------------------ writing
// A lane takes PC pieces of 16 bytes (D is a multiple of that many elements),
// LANES lanes a row: the power of two that covers it (4 at least).
template <typename T, bool E4M3, int LANES, int PC>
__global__ void __launch_bounds__(kWarps * 32, 12) cache_write_vec(const CacheRowsParams p) {
  constexpr int VEC = 16 / sizeof(T), EL = VEC * PC;  // elements of a piece, of a lane
  using C = typename std::conditional<E4M3, uint8_t, T>::type;
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  check_offsets(p);
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  constexpr int per = 32 / LANES;  // heads at once
  const int sub = lane / LANES, dl = lane % LANES * EL;
  const bool in_row = dl < p.c.D && JVP_CHECK(dl + EL <= p.c.D, p.c.status, kChkGlobalCol);
  const T* const ks = static_cast<const T*>(p.k) + r * p.srk.n + dl;
  const T* const vs = static_cast<const T*>(p.v) + r * p.srv.n + dl;
  C* const kd = static_cast<C*>(p.c.k) + page * p.c.sk.b + row * p.c.sk.n + dl;
  C* const vd = static_cast<C*>(p.c.v) + page * p.c.sv.b + row * p.c.sv.n + dl;
  const long long scale_at = static_cast<long long>(page) * p.c.Hkv * p.c.page_size + row;
  constexpr int UN = 4 / PC;  // heads of one lane group in flight
  for (int i0 = 0; i0 < 2 * p.c.Hkv; i0 += per * UN) {
    uint4 x[UN][PC];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const HeadRow at = head_row(p.c, i0 + u * per + sub, in_row);
      const T* src = at.v ? vs + at.h * p.srv.h : ks + at.h * p.srk.h;
#pragma unroll
      for (int i = 0; i < PC; ++i)
        x[u][i] = at.on ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (i0 + u * per >= 2 * p.c.Hkv) break;  // uniform over the warp
      const HeadRow at = head_row(p.c, i0 + u * per + sub, in_row);
      C* dst = at.v ? vd + at.h * p.c.sv.h : kd + at.h * p.c.sk.h;
      if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < PC; ++i)
          if (at.on) reinterpret_cast<uint4*>(dst)[i] = x[u][i];
      } else {
        const unsigned sb = scale_byte(group_top<LANES>(ks, x[u]));
        const float inv = __uint_as_float((254u - sb) << 23);  // 2^-e, e = sb - 127
        constexpr int W = 4 / sizeof(T);
        uint32_t c[PC * W];
#pragma unroll
        for (int i = 0; i < PC; ++i)
          encode<T>(x[u][i], inv, *reinterpret_cast<uint32_t(*)[W]>(&c[i * W]));
        if (at.on) {
          put_words(dst, c);
          if (dl == 0)
            (at.v ? p.c.v_scale : p.c.k_scale)[scale_at + at.h * p.c.page_size] =
                static_cast<uint8_t>(sb);
        }
      }
    }
  }
}

// Any D and alignment: one head of a row at a time, lane-strided elements.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_write_any(const CacheRowsParams p) {
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  check_offsets(p);
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  for (int hw = 0; hw < 2 * p.c.Hkv; ++hw) {
    const int h = hw >> 1, w = hw & 1;
    const Strides& ss = w ? p.srv : p.srk;
    const Strides& sc = w ? p.c.sv : p.c.sk;
    const T* src = static_cast<const T*>(w ? p.v : p.k) + r * ss.n + h * ss.h;
    void* cache = w ? p.c.v : p.c.k;
    const long long at = page * sc.b + h * sc.h + row * sc.n;
    if constexpr (!E4M3) {
      for (int d = lane; d < p.c.D; d += 32) static_cast<T*>(cache)[at + d] = src[d];
    } else {
      float top = 0.f;
      for (int d = lane; d < p.c.D; d += 32) top = fmaxf(top, fabsf(Rows<T>::get(src[d])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const unsigned sb = scale_byte(top);
      const float inv = __uint_as_float((254u - sb) << 23);
      for (int d = lane; d < p.c.D; d += 32)
        static_cast<uint8_t*>(cache)[at + d] =
            static_cast<uint8_t>(to_e4m3x2(Rows<T>::get(src[d]) * inv, 0.f) & 0xFFu);
      if (lane == 0)
        (w ? p.c.v_scale : p.c.k_scale)[(static_cast<long long>(page) * p.c.Hkv + h) *
                                            p.c.page_size + row] = static_cast<uint8_t>(sb);
    }
  }
}

// ------------------------------------------------------------------ reading
template <typename T, bool E4M3, int LANES>
__global__ void __launch_bounds__(kWarps * 32) cache_read_vec(const CacheRowsParams p) {
  constexpr int VEC = 16 / sizeof(T);
  using C = typename std::conditional<E4M3, uint8_t, T>::type;
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  check_offsets(p);
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  constexpr int per = 32 / LANES;
  const int sub = lane / LANES, dl = lane % LANES * VEC;
  const bool in_row = dl < p.c.D && JVP_CHECK(dl + VEC <= p.c.D, p.c.status, kChkGlobalCol);
  const C* const ks = static_cast<const C*>(p.c.k) + page * p.c.sk.b + row * p.c.sk.n + dl;
  const C* const vs = static_cast<const C*>(p.c.v) + page * p.c.sv.b + row * p.c.sv.n + dl;
  T* const kd = const_cast<T*>(static_cast<const T*>(p.k)) + r * p.srk.n + dl;
  T* const vd = const_cast<T*>(static_cast<const T*>(p.v)) + r * p.srv.n + dl;
  const long long scale_at = static_cast<long long>(page) * p.c.Hkv * p.c.page_size + row;
  constexpr int UN = 4;
  constexpr int W = (E4M3 ? 4 : 16) / (E4M3 ? sizeof(T) : 4);  // 32-bit words of a lane's part
  for (int i0 = 0; i0 < 2 * p.c.Hkv; i0 += per * UN) {
    uint32_t x[UN][W];
    unsigned sb[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const HeadRow at = head_row(p.c, i0 + u * per + sub, in_row);
      if (!at.on) continue;
      const C* src = at.v ? vs + at.h * p.c.sv.h : ks + at.h * p.c.sk.h;
      get_words(reinterpret_cast<const uint8_t*>(src), x[u]);
      if constexpr (E4M3)
        sb[u] = __ldg((at.v ? p.c.v_scale : p.c.k_scale) + scale_at + at.h * p.c.page_size);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const HeadRow at = head_row(p.c, i0 + u * per + sub, in_row);
      if (!at.on) continue;
      T* dst = at.v ? vd + at.h * p.srv.h : kd + at.h * p.srk.h;
      if constexpr (E4M3)
        *reinterpret_cast<uint4*>(dst) = decode<T>(x[u], scale_value(sb[u]));
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
    }
  }
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_any(const CacheRowsParams p) {
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  check_offsets(p);
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  for (int hw = 0; hw < 2 * p.c.Hkv; ++hw) {
    const int h = hw >> 1, w = hw & 1;
    const Strides& sr = w ? p.srv : p.srk;
    const Strides& sc = w ? p.c.sv : p.c.sk;
    T* dst = const_cast<T*>(static_cast<const T*>(w ? p.v : p.k)) + r * sr.n + h * sr.h;
    const void* cache = w ? p.c.v : p.c.k;
    const long long at = page * sc.b + h * sc.h + row * sc.n;
    float s = 1.f;
    if (E4M3)
      s = scale_value((w ? p.c.v_scale : p.c.k_scale)[(static_cast<long long>(page) * p.c.Hkv + h) *
                                                          p.c.page_size + row]);
    for (int d = lane; d < p.c.D; d += 32) {
      if constexpr (E4M3) {
        const uint32_t h2 = e4m3x2_to_half2(static_cast<const uint8_t*>(cache)[at + d]);
        dst[d] = Rows<T>::put(__half22float2(*reinterpret_cast<const __half2*>(&h2)).x * s);
      } else {
        dst[d] = static_cast<const T*>(cache)[at + d];
      }
    }
  }
}

template <typename T, bool E4M3, bool WRITE, int LANES, int PC>
void launch_vec(unsigned grid, const CacheRowsParams& p, cudaStream_t stream) {
  if constexpr (LANES * PC < (sizeof(T) == 4 ? 32 : 16)) {  // D <= 128
    if (p.c.D > LANES * PC * static_cast<int>(16 / sizeof(T)))
      return launch_vec<T, E4M3, WRITE, LANES * 2, PC>(grid, p, stream);
  }
  if constexpr (WRITE) cache_write_vec<T, E4M3, LANES, PC><<<grid, kWarps * 32, 0, stream>>>(p);
  else cache_read_vec<T, E4M3, LANES><<<grid, kWarps * 32, 0, stream>>>(p);
}

template <typename T, bool E4M3, bool WRITE>
cudaError_t launch(const CacheRowsParams& p, cudaStream_t stream) {
  // a warp for each row, a thread for each sequence's offsets
  const long long rows = (p.T + kWarps - 1) / kWarps;
  const long long offsets = p.cu ? (p.c.B + kWarps * 32 - 1ll) / (kWarps * 32) : 0;
  const unsigned grid = static_cast<unsigned>(rows > offsets ? rows : offsets);
  if (p.vec) {
    // Two pieces a lane where the cost is instructions, in writing e4m3 rows,
    // and they fit; reading them that way took 67.7 us against 60.7.
    if constexpr (WRITE && E4M3) {
      if (p.vec == 2) {
        launch_vec<T, E4M3, WRITE, 4, 2>(grid, p, stream);
        return cudaGetLastError();
      }
    }
    launch_vec<T, E4M3, WRITE, 4, 1>(grid, p, stream);
  } else {
    if constexpr (WRITE) cache_write_any<T, E4M3><<<grid, kWarps * 32, 0, stream>>>(p);
    else cache_read_any<T, E4M3><<<grid, kWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <bool WRITE>
cudaError_t dispatch(DType dt, bool e4m3, const CacheRowsParams& p, cudaStream_t stream) {
  switch (dt) {
    case kF32: return e4m3 ? launch<float, true, WRITE>(p, stream) : launch<float, false, WRITE>(p, stream);
    case kF16: return e4m3 ? launch<__half, true, WRITE>(p, stream) : launch<__half, false, WRITE>(p, stream);
    case kBF16:
      return e4m3 ? launch<__nv_bfloat16, true, WRITE>(p, stream)
                  : launch<__nv_bfloat16, false, WRITE>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_write(DType dt, bool e4m3, const CacheRowsParams& p, cudaStream_t stream) {
  return dispatch<true>(dt, e4m3, p, stream);
}
cudaError_t launch_cache_read(DType dt, bool e4m3, const CacheRowsParams& p, cudaStream_t stream) {
  return dispatch<false>(dt, e4m3, p, stream);
}

}  // namespace jvp
