// paged.cuh -- addressing of a paged key-value cache: which page and row hold
// a position of a sequence, with every index that comes from device memory
// checked before it is used.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "serve_internal.h"

namespace jvp {

// Keys a sequence can have: its length, limited to what its pages can hold.
// *bad is set for a length outside [0, max_pages * page_size].
__device__ __forceinline__ int clamp_len(const PagedCache& c, int len, bool* bad) {
  const long long most = static_cast<long long>(c.max_pages) * c.page_size;
  if (len < 0 || len > most) {
    *bad = true;
    return len < 0 ? 0 : static_cast<int>(most);
  }
  return len;
}

// Place of a position within its sequence's pages: index into the block table
// row and row of the page.
__device__ __forceinline__ void split_position(const PagedCache& c, int pos, int* entry,
                                               int* row) {
  if (c.page_shift >= 0) {
    *entry = pos >> c.page_shift;
    *row = pos & (c.page_size - 1);
  } else {
    *entry = pos / c.page_size;
    *row = pos - *entry * c.page_size;
  }
}

// Page of a block table entry, or -1 (recorded in the status word) where the
// entry names no page of the cache.  entry must be in [0, max_pages).
__device__ __forceinline__ int page_of(const PagedCache& c, int b, int entry) {
  const int page = __ldg(c.table + b * c.table_stride + entry);
  if (page < 0 || page >= c.pages) {
    atomicOr(c.status, kStatusIndex);
    return -1;
  }
  return page;
}

// 2^(byte - 127), exact for every byte (0 is the subnormal 2^-127, which the
// fp32 arithmetic here keeps; 255 never occurs in a written cache and reads as
// infinity).
__device__ __forceinline__ float scale_value(unsigned byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Two e4m3 codes (low and high byte of x) as fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
  return r;
}

// Four e4m3 codes as two pairs of fp16 values (codes 0, 1 and codes 2, 3).
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// Looks at the offsets of sequence i, if there is one.
__device__ __forceinline__ void check_sequence_offsets(const PagedCache& c, const int* cu,
                                                       long long T, long long i) {
  if (!cu || i >= c.B) return;
  const int r0 = __ldg(cu + i), r1 = __ldg(cu + i + 1);
  if (r0 < 0 || r1 < r0 || r1 > T) atomicOr(c.status, kStatusIndex);
}

// Where row r of T packed rows lives in the cache (start: position of each
// sequence's first row, nullptr: 0; cu: nullptr for one row per sequence), and its
// position: false if it belongs to no sequence, or (recorded in the status
// word) its sequence's offsets or its place are out of range.
__device__ __forceinline__ bool locate_row(const PagedCache& c, const int* cu, const int* start,
                                           long long T, long long r, int* page, int* row,
                                           int* position) {
  int b;
  long long first;
  if (cu) {
    // last b with cu[b] <= r
    int lo = -1, hi = c.B;  // cu[lo] <= r < cu[hi], the ends taken as given
    while (hi - lo > 1) {
      const int mid = lo + ((hi - lo) >> 1);  // (lo + hi may pass 2^31)
      if (__ldg(cu + mid) <= r) lo = mid;
      else hi = mid;
    }
    // rows before the first sequence and behind the last are in none
    if (lo < 0) return false;
    b = lo;
    first = __ldg(cu + b);
    const int end = __ldg(cu + b + 1);
    if (end <= r || first < 0 || end > T) return false;  // (check_sequence_offsets records what is wrong)
  } else {
    b = static_cast<int>(r);
    first = r;
  }
  const long long pos = (start ? static_cast<long long>(__ldg(start + b)) : 0ll) + (r - first);
  const long long most = static_cast<long long>(c.max_pages) * c.page_size;
  if (pos < 0 || pos >= most) {
    atomicOr(c.status, kStatusIndex);
    return false;
  }
  *position = static_cast<int>(pos);
  int entry;
  split_position(c, static_cast<int>(pos), &entry, row);
  *page = page_of(c, b, entry);
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

}  // namespace jvp
