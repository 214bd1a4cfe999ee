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

}  // namespace jvp
