// serve_checks.h -- argument checks and descriptions that the serving entry
// points share.
#pragma once

#include <cudaTypedefs.h>

#include "serve_internal.h"

namespace jvp {

constexpr int64_t kMax = (1ll << 31) - 1;
// Positions, rows and sequences: below this the end of a tile, or of a thread's
// share of them, is a 32-bit number too.
constexpr int64_t kMaxRows = (1ll << 31) - 1024;

inline bool aligned_to(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int64_t elem_bytes(int dt) { return dt == JVP_E4M3 ? 1 : dt == JVP_F32 ? 4 : 2; }
inline bool tensor_type(int dt) { return dt == JVP_F32 || dt == JVP_F16 || dt == JVP_BF16; }

// Strides with those of size-1 dimensions (never used) set to 0.
inline Strides used(const jvp_strides_t& s, int64_t b, int64_t h, int64_t n) {
  return Strides{b > 1 ? s.b : 0, h > 1 ? s.h : 0, n > 1 ? s.n : 0};
}
inline bool multiple(const Strides& s, int64_t m) { return s.b % m == 0 && s.h % m == 0 && s.n % m == 0; }

inline jvp_status_t check_strides(const jvp_strides_t& s, const char* what_d, const char* what_neg) {
  if (s.d != 1) return api_fail(JVP_ERR_INVALID_ARG, what_d);
  if (s.b < 0 || s.h < 0 || s.n < 0) return api_fail(JVP_ERR_INVALID_ARG, what_neg);
  return JVP_OK;
}

// Why a window and its sinks are refused, or nullptr.
inline const char* bad_window(int64_t window, int64_t sinks) {
  return window <= 0 ? "window must be positive" : sinks < 0 ? "negative number of sinks" : nullptr;
}

// Sizes, types and strides of a cache description (no pointers).
inline jvp_status_t check_cache(const jvp_cache_t* c, bool written) {
  if (!c) return api_fail(JVP_ERR_INVALID_ARG, "cache is NULL");
  if (c->pages < 0 || c->Hkv < 0 || c->B < 0 || c->max_pages < 0 || c->table_stride < 0)
    return api_fail(JVP_ERR_INVALID_ARG, "negative size in the cache description");
  if (c->page_size <= 0) return api_fail(JVP_ERR_INVALID_ARG, "page_size must be positive");
  if (c->D <= 0) return api_fail(JVP_ERR_INVALID_ARG, "D must be positive");
  if (c->D > 128) return api_fail(JVP_ERR_UNSUPPORTED, "D > 128 is not supported");
  if (!tensor_type(c->dtype) && c->dtype != JVP_E4M3)
    return api_fail(JVP_ERR_INVALID_ARG, "unknown cache dtype");
  if (c->pages > kMax || c->Hkv > kMax || c->B > kMaxRows || c->max_pages > kMax ||
      c->page_size > kMax || c->max_pages * c->page_size > kMaxRows)
    return api_fail(JVP_ERR_UNSUPPORTED,
                    "a size of the cache exceeds 2^31 - 1, or B or max_pages * page_size 2^31 - 1024");
  if (c->B > 1 && c->table_stride < c->max_pages)
    return api_fail(JVP_ERR_INVALID_ARG, "table_stride is less than max_pages");
  for (const jvp_strides_t* s : {&c->k_strides, &c->v_strides}) {
    const jvp_status_t st = check_strides(*s, "innermost (d) stride of the cache must be 1",
                                          "negative cache stride");
    if (st != JVP_OK) return st;
    if (written && ((c->pages > 1 && s->b == 0) || (c->Hkv > 1 && s->h == 0) ||
                    (c->page_size > 1 && s->n == 0)))
      return api_fail(JVP_ERR_INVALID_ARG, "a written cache must not have a stride of 0");
  }
  return JVP_OK;
}

// Pointers of a cache, once the sizes are known to be good.
inline jvp_status_t check_cache_ptrs(const jvp_cache_t* c, const void* k, const void* v, const void* ks,
                              const void* vs, const int32_t* table) {
  if (c->pages > 0 && c->Hkv > 0) {
    if (!k || !v) return api_fail(JVP_ERR_INVALID_ARG, "cache pointer is NULL");
    if (c->dtype == JVP_E4M3 && (!ks || !vs))
      return api_fail(JVP_ERR_INVALID_ARG, "an e4m3 cache needs k_scale and v_scale");
  }
  if (!aligned_to(k, elem_bytes(c->dtype)) || !aligned_to(v, elem_bytes(c->dtype)))
    return api_fail(JVP_ERR_ALIGNMENT, "cache not aligned to its element size");
  if (!table && c->B > 0 && c->max_pages > 0)
    return api_fail(JVP_ERR_INVALID_ARG, "block_table is NULL");
  if (!aligned_to(table, 4)) return api_fail(JVP_ERR_ALIGNMENT, "block_table is not 4-byte aligned");
  return JVP_OK;
}

inline PagedCache describe(const jvp_cache_t* c, const void* k, const void* v, const uint8_t* ks,
                    const uint8_t* vs, const int32_t* table, unsigned int* status) {
  PagedCache p{};
  p.pages = static_cast<int>(c->pages), p.Hkv = static_cast<int>(c->Hkv);
  p.page_size = static_cast<int>(c->page_size), p.D = static_cast<int>(c->D);
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (c->page_size == (1ll << s)) p.page_shift = s;
  p.B = static_cast<int>(c->B), p.max_pages = static_cast<int>(c->max_pages);
  p.table_stride = c->table_stride;
  p.table = table;
  p.k = const_cast<void*>(k), p.v = const_cast<void*>(v);
  p.sk = used(c->k_strides, c->pages, c->Hkv, c->page_size);
  p.sv = used(c->v_strides, c->pages, c->Hkv, c->page_size);
  p.k_scale = const_cast<uint8_t*>(ks), p.v_scale = const_cast<uint8_t*>(vs);
  p.status = status;
  return p;
}

// Tiled map of a packed 16-bit tensor: `inner`, `mid` and `outer` are (D and)
// two dimensions with their strides in elements, the box {64, bmid, bouter},
// 128-byte swizzle.  False if the layout cannot be described.
inline bool encode_packed(CUtensorMap* map, int dt, const void* ptr, int64_t D, int64_t mid,
                   int64_t mid_stride, int64_t outer, int64_t outer_stride, int bmid, int bouter) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(api_tensor_map_encoder());
  if (!enc || !aligned_to(ptr, 16)) return false;
  // a size-1 dimension's stride is never used; give it a well-formed value
  if (mid == 1) mid_stride = D;
  if (outer == 1) outer_stride = D;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(mid),
                        static_cast<cuuint64_t>(outer), 1};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(mid_stride * 2),
                           static_cast<cuuint64_t>(outer_stride * 2), static_cast<cuuint64_t>(D * 2)};
  for (auto s : strides)
    if (s == 0 || s % 16 != 0 || s >= (1ull << 40)) return false;
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(bmid), static_cast<cuuint32_t>(bouter), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, dt == JVP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             4, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace jvp
