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
// a group of lanes takes one head with 16 bytes per lane of the 16- or 32-bit
// side, and the heads are unrolled so that several loads are in flight.
#include <cmath>

#include "paged.cuh"

namespace jvp {
namespace {

constexpr int kWarps = 8;  // rows per block

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

// Where row r of the packed tensors lives in the cache: false if it belongs to
// no sequence, or (recorded in the status word) its place is out of range.
__device__ __forceinline__ bool locate(const CacheRowsParams& p, long long r, int* page, int* row) {
  int b;
  long long first;
  if (p.cu) {
    // last b with cu[b] <= r
    int lo = -1, hi = p.c.B;  // cu[lo] <= r < cu[hi], the ends taken as given
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= r) lo = mid;
      else hi = mid;
    }
    // rows before the first sequence and behind the last are in none
    if (lo < 0 || __ldg(p.cu + p.c.B) <= r) return false;
    b = lo;
    first = __ldg(p.cu + b);
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

// ------------------------------------------------------------------ writing
// VEC elements of type T are 16 bytes; D is a multiple of VEC.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, 4) cache_write_vec(const CacheRowsParams p, int lanes) {
  constexpr int VEC = 16 / sizeof(T);
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  // group of `lanes` lanes (a power of two) per head, 32 / lanes heads at once
  const int per = 32 / lanes, sub = lane / lanes, dl = (lane & (lanes - 1)) * VEC;
  const bool in_row = dl < p.c.D;
  constexpr int UN = E4M3 ? 2 : 4;  // heads of one lane group in flight, for K and V each
  for (int h0 = 0; h0 < p.c.Hkv; h0 += per * UN) {
    uint4 x[2][UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int h = h0 + u * per + sub;
      const bool on = h < p.c.Hkv && in_row;
      const T* ks = static_cast<const T*>(p.k) + r * p.srk.n + h * p.srk.h + dl;
      const T* vs = static_cast<const T*>(p.v) + r * p.srv.n + h * p.srv.h + dl;
      x[0][u] = on ? __ldg(reinterpret_cast<const uint4*>(ks)) : make_uint4(0, 0, 0, 0);
      x[1][u] = on ? __ldg(reinterpret_cast<const uint4*>(vs)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (h0 + u * per >= p.c.Hkv) break;  // uniform over the warp
      const int h = h0 + u * per + sub;
      const bool on = h < p.c.Hkv && in_row;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const Strides& sc = w ? p.c.sv : p.c.sk;
        const long long at = page * sc.b + h * sc.h + row * sc.n + dl;
        void* cache = w ? p.c.v : p.c.k;
        if constexpr (!E4M3) {
          if (on) *reinterpret_cast<uint4*>(static_cast<T*>(cache) + at) = x[w][u];
        } else {
          const T* e = reinterpret_cast<const T*>(&x[w][u]);
          float f[VEC], top = 0.f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            f[i] = Rows<T>::get(e[i]);
            top = fmaxf(top, fabsf(f[i]));
          }
          for (int o = lanes >> 1; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const unsigned sb = scale_byte(top);
          const float inv = __uint_as_float((254u - sb) << 23);  // 2^-e, e = sb - 127
          if (on) {
            uint32_t c[VEC / 4];
#pragma unroll
            for (int i = 0; i < VEC; i += 4)
              c[i / 4] = to_e4m3x2(f[i] * inv, f[i + 1] * inv) |
                         (static_cast<uint32_t>(to_e4m3x2(f[i + 2] * inv, f[i + 3] * inv)) << 16);
            uint8_t* dst = static_cast<uint8_t*>(cache) + at;
            if constexpr (VEC == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
            else *reinterpret_cast<uint32_t*>(dst) = c[0];
            if (dl == 0) {
              uint8_t* scale = w ? p.c.v_scale : p.c.k_scale;
              scale[(static_cast<long long>(page) * p.c.Hkv + h) * p.c.page_size + row] =
                  static_cast<uint8_t>(sb);
            }
          }
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
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_vec(const CacheRowsParams p, int lanes) {
  constexpr int VEC = 16 / sizeof(T);
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= p.T) return;
  int page, row;
  if (!locate(p, r, &page, &row)) return;
  const int per = 32 / lanes, sub = lane / lanes, dl = (lane & (lanes - 1)) * VEC;
  const bool in_row = dl < p.c.D;
  constexpr int UN = 4;
  for (int h0 = 0; h0 < p.c.Hkv; h0 += per * UN) {
    uint4 x[2][UN];
    unsigned sb[2][UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int h = h0 + u * per + sub;
      const bool on = h < p.c.Hkv && in_row;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const Strides& sc = w ? p.c.sv : p.c.sk;
        const void* cache = w ? p.c.v : p.c.k;
        const long long at = page * sc.b + h * sc.h + row * sc.n + dl;
        x[w][u] = make_uint4(0, 0, 0, 0);
        if (on) {
          if constexpr (!E4M3) {
            x[w][u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(cache) + at));
          } else {
            const uint8_t* src = static_cast<const uint8_t*>(cache) + at;
            if constexpr (VEC == 8) {
              const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
              x[w][u].x = c.x, x[w][u].y = c.y;
            } else {
              x[w][u].x = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
            sb[w][u] = __ldg((w ? p.c.v_scale : p.c.k_scale) +
                             (static_cast<long long>(page) * p.c.Hkv + h) * p.c.page_size + row);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int h = h0 + u * per + sub;
      if (h >= p.c.Hkv || !in_row) continue;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const Strides& sr = w ? p.srv : p.srk;
        T* dst = const_cast<T*>(static_cast<const T*>(w ? p.v : p.k)) + r * sr.n + h * sr.h + dl;
        if constexpr (E4M3) {
          const float s = scale_value(sb[w][u]);
          const uint32_t c[2] = {x[w][u].x, x[w][u].y};
          T e[VEC];
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const uint32_t h2 = e4m3x2_to_half2((c[i / 4] >> (8 * (i & 2))) & 0xFFFFu);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            e[i] = Rows<T>::put(f.x * s);
            e[i + 1] = Rows<T>::put(f.y * s);
          }
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(e);
        } else {
          *reinterpret_cast<uint4*>(dst) = x[w][u];
        }
      }
    }
  }
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_any(const CacheRowsParams p) {
  const long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
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

template <typename T, bool E4M3, bool WRITE>
cudaError_t launch(const CacheRowsParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.T + kWarps - 1) / kWarps);
  if (p.vec) {
    const int need = p.c.D / static_cast<int>(16 / sizeof(T));
    int lanes = 1;
    while (lanes < need) lanes *= 2;
    if (WRITE) cache_write_vec<T, E4M3><<<grid, kWarps * 32, 0, stream>>>(p, lanes);
    else cache_read_vec<T, E4M3><<<grid, kWarps * 32, 0, stream>>>(p, lanes);
  } else {
    if (WRITE) cache_write_any<T, E4M3><<<grid, kWarps * 32, 0, stream>>>(p);
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
