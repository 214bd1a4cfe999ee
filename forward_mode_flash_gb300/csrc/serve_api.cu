// serve_api.cu -- entry points of the attention over packed prompts, the paged
// key-value cache and the single-token attention over it: argument checks,
// path selection and launch descriptions.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "serve_checks.h"

namespace jvp {
namespace {

jvp_status_t cache_rows(bool write, const jvp_cache_t* c, jvp_dtype_t dtype, int64_t T,
                        const void* k, const void* v, const jvp_strides_t* strides,
                        const int32_t* table, const int32_t* start, const int32_t* cu,
                        const void* kc, const void* vc, const uint8_t* ks, const uint8_t* vs,
                        void* stream) {
  api_set_path(0);
  jvp_status_t st = check_cache(c, write);
  if (st != JVP_OK) return st;
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  if (c->dtype != JVP_E4M3 && c->dtype != dtype)
    return api_fail(JVP_ERR_INVALID_ARG, "the rows must have the cache's dtype (or the cache e4m3)");
  if (T < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative T");
  if (T > kMax) return api_fail(JVP_ERR_UNSUPPORTED, "T exceeds 2^31 - 1");
  // (the kernels walk the heads of K and V as one list, up to 32 at a time)
  if (c->Hkv > kMax / 2 - 64) return api_fail(JVP_ERR_UNSUPPORTED, "Hkv exceeds 2^30 - 65");
  if (!cu && T != c->B)
    return api_fail(JVP_ERR_INVALID_ARG, "without cu_seqlens there must be one row per sequence");
  if (!strides) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  for (int i = 0; i < 2; ++i) {
    st = check_strides(strides[i], "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
    if (!write && ((T > 1 && strides[i].n == 0) || (c->Hkv > 1 && strides[i].h == 0)))
      return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  }
  if (T == 0 || c->B == 0 || c->Hkv == 0) return api_ok();
  if (!k || !v) return api_fail(JVP_ERR_INVALID_ARG, "k or v is NULL");
  const int64_t e = elem_bytes(dtype);
  if (!aligned_to(k, e) || !aligned_to(v, e))
    return api_fail(JVP_ERR_ALIGNMENT, "k or v not aligned to its element size");
  if (!aligned_to(start, 4) || !aligned_to(cu, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "start_pos or cu_seqlens not 4-byte aligned");
  st = check_cache_ptrs(c, kc, vc, ks, vs, table);
  if (st != JVP_OK) return st;
  int sms = 0;
  unsigned int* status = nullptr;
  st = api_device(&sms, &status);
  if (st != JVP_OK) return st;

  CacheRowsParams p{};
  p.c = describe(c, kc, vc, ks, vs, table, status);
  p.T = T;
  p.cu = cu, p.start = start;
  p.k = k, p.v = v;
  p.srk = used(strides[0], 0, c->Hkv, T), p.srv = used(strides[1], 0, c->Hkv, T);
  // 16 bytes of packed rows per access and the same elements of the cache, or
  // (an e4m3 cache) two such pieces per lane and their elements of the cache
  const int64_t ce = elem_bytes(c->dtype);
  auto fits = [&](int64_t el) {
    return c->D % el == 0 && aligned_to(kc, el * ce) && aligned_to(vc, el * ce) &&
           multiple(p.c.sk, el) && multiple(p.c.sv, el);
  };
  const int64_t vec = 16 / e;
  // (the kernel of 16-byte accesses has 32-bit offsets of the scales within a
  // page: with 64-bit ones it took 3 to 5 % longer)
  const bool scales_fit = c->dtype != JVP_E4M3 || c->page_size <= kMax / c->Hkv;
  p.vec = scales_fit && aligned_to(k, 16) && aligned_to(v, 16) && multiple(p.srk, vec) &&
                  multiple(p.srv, vec) && fits(vec)
              ? (ce == 1 && fits(2 * vec) ? 2 : 1)
              : 0;
  const bool e4m3 = c->dtype == JVP_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = write ? launch_cache_write(static_cast<DType>(dtype), e4m3, p, s)
                                : launch_cache_read(static_cast<DType>(dtype), e4m3, p, s);
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(2);
  return api_ok();
}

// CTAs of the single-token attention and the query heads each takes.
struct DecodePlan {
  int heads_per_block = 0, head_blocks = 0, grid = 0, direct = 0;
  size_t bytes = 0, at_o = 0, at_cta = 0;  // workspace: lse, partial outputs, CTAs of segments
};
// window: 0 for none.
DecodePlan plan_decode(const jvp_cache_t* c, int64_t H, bool tc, int num_sms, int64_t window,
                       int64_t sinks) {
  DecodePlan d;
  const int D = static_cast<int>(c->D), group = static_cast<int>(H / c->Hkv);
  d.heads_per_block = decode_heads_per_block(tc, group);
  d.head_blocks = (group + d.heads_per_block - 1) / d.heads_per_block;
  const int64_t most = c->max_pages * c->page_size;
  const int64_t wave =
      static_cast<int64_t>(num_sms) *
      (tc ? decode_ctas_per_sm(D, d.heads_per_block / 8, c->dtype == JVP_E4M3)
          : decode_simt_ctas_per_sm(d.heads_per_block));
  const int tile = decode_tile(tc, D, c->dtype == JVP_E4M3);
  int64_t tiles = (most + tile - 1) / tile;
  // B * Hkv * head_blocks <= B * H <= 2^31 - 1 (checked by the caller), tiles < 2^31
  const int64_t segments = c->B * c->Hkv * d.head_blocks;
  int direct = kDecodeDirectTiles;
  if (window > 0) {  // (its keys begin anywhere in a tile)
    const int64_t seen = (window + tile - 2) / tile + 1 + (sinks + tile - 1) / tile;
    if (seen < tiles) {
      tiles = seen;
      if (tc)
        direct = decode_window_direct(D, c->dtype == JVP_E4M3, d.heads_per_block,
                                      segments >= num_sms);
    }
  }
  if (tiles > 0 && tiles <= direct) {
    d.grid = static_cast<int>(segments), d.direct = 1;
    return d;
  }
  d.grid = static_cast<int>(std::min<int64_t>(wave, tiles ? (segments > wave ? wave : segments * tiles) : 0));
  const size_t slots = static_cast<size_t>(d.grid) * 2 * d.heads_per_block;
  if (d.grid > 0) {
    d.at_o = (slots * 4 + 255) & ~static_cast<size_t>(255);
    d.at_cta = d.at_o + slots * (D > 64 ? 128 : 64) * 4;
    d.bytes = d.at_cta + static_cast<size_t>(segments) * 8;
  }
  return d;
}

jvp_status_t check_decode(const jvp_cache_t* c, int64_t H, int dtype) {
  const jvp_status_t st = check_cache(c, false);
  if (st != JVP_OK) return st;
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  if (c->dtype != JVP_E4M3 && c->dtype != dtype)
    return api_fail(JVP_ERR_INVALID_ARG, "q must have the cache's dtype (or the cache e4m3)");
  if (H < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative H");
  if (H > kMax || c->B * H > kMax)
    return api_fail(JVP_ERR_UNSUPPORTED, "problem too large for one launch");
  if (c->Hkv == 0 ? H > 0 : H % c->Hkv != 0)
    return api_fail(JVP_ERR_INVALID_ARG, "H must be a multiple of Hkv (grouped-query attention)");
  return JVP_OK;
}

// window: 0 for none.
jvp_status_t decode(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype, const void* q,
                    const jvp_strides_t* q_strides, const void* k_cache, const void* v_cache,
                    const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                    const int32_t* seq_lens, int64_t window, int64_t sinks, float scale, void* o,
                    const jvp_strides_t* o_strides, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  api_set_path(0);
  jvp_status_t st = check_decode(cache, H, dtype);
  if (st != JVP_OK) return st;
  if (!std::isfinite(scale)) return api_fail(JVP_ERR_INVALID_ARG, "scale is not finite");
  if (!q_strides || !o_strides) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  const int64_t B = cache->B, D = cache->D;
  for (const jvp_strides_t* s : {q_strides, o_strides}) {
    st = check_strides(*s, "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
  }
  if ((B > 1 && o_strides->b == 0) || (H > 1 && o_strides->h == 0))
    return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  if (B == 0 || H == 0) return api_ok();
  if (!q || !o || !seq_lens) return api_fail(JVP_ERR_INVALID_ARG, "q, o or seq_lens is NULL");
  const int64_t e = elem_bytes(dtype), ce = elem_bytes(cache->dtype);
  if (!aligned_to(q, e) || !aligned_to(o, e))
    return api_fail(JVP_ERR_ALIGNMENT, "q or o not aligned to its element size");
  if (!aligned_to(lse, 4) || !aligned_to(seq_lens, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "lse or seq_lens not 4-byte aligned");
  st = check_cache_ptrs(cache, k_cache, v_cache, k_scale, v_scale, block_table);
  if (st != JVP_OK) return st;
  int sms = 0;
  unsigned int* status = nullptr;
  st = api_device(&sms, &status);
  if (st != JVP_OK) return st;

  DecodeParams p{};
  p.c = describe(cache, k_cache, v_cache, k_scale, v_scale, block_table, status);
  p.H = static_cast<int>(H), p.group = static_cast<int>(H / cache->Hkv);
  p.lens = seq_lens;
  p.q = q, p.sq = used(*q_strides, B, H, 0);
  p.o = o, p.so = used(*o_strides, B, H, 0);
  p.lse = lse;
  p.scale_log2 = scale * 1.4426950408889634f;
  const bool e4m3 = cache->dtype == JVP_E4M3;
  const bool tc = e == 2 && D % (e4m3 ? 16 : 8) == 0 && aligned_to(q, 8) && multiple(p.sq, 4) &&
                  aligned_to(k_cache, 16) && aligned_to(v_cache, 16) &&
                  multiple(p.c.sk, 16 / ce) && multiple(p.c.sv, 16 / ce);
  const bool vec = D % 4 == 0 && aligned_to(k_cache, 4 * ce) && aligned_to(v_cache, 4 * ce) &&
                   multiple(p.c.sk, 4) && multiple(p.c.sv, 4);
  const DecodePlan d = plan_decode(cache, H, tc, sms, window, sinks);
  if (d.bytes > 0 && (!workspace || workspace_bytes < d.bytes))
    return api_fail(JVP_ERR_WORKSPACE,
                    "workspace is NULL or smaller than jvp_attn_decode_workspace_size()");
  if (!aligned_to(workspace, 16)) return api_fail(JVP_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  p.o_vec = aligned_to(o, 16) && multiple(p.so, 8);
  p.head_blocks = d.head_blocks, p.grid = d.grid, p.direct = d.direct;
  if (d.bytes > 0) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.ws_lse = reinterpret_cast<float*>(ws);
    p.ws_o = reinterpret_cast<float*>(ws + d.at_o);
    p.ws_cta = reinterpret_cast<int2*>(ws + d.at_cta);
  }
  p.window = static_cast<int>(window), p.sinks = static_cast<int>(sinks);
  const cudaError_t err = (window > 0 ? launch_decode_window : launch_decode)(
      static_cast<DType>(dtype), e4m3, tc, vec, p, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(tc ? 1 : 2);
  return api_ok();
}

}  // namespace
}  // namespace jvp

extern "C" {

jvp_status_t jvp_attn_fwd_packed(const jvp_packed_shape_t* shape, jvp_dtype_t dtype, const void* q,
                                 const void* k, const void* v, const jvp_strides_t* in_strides,
                                 const int32_t* cu_seqlens, int causal, float scale, void* o,
                                 const jvp_strides_t* out_strides, float* lse, void* stream) {
  using namespace jvp;
  api_set_path(0);
  if (!shape) return api_fail(JVP_ERR_INVALID_ARG, "shape is NULL");
  const int64_t T = shape->T, B = shape->B, H = shape->H, D = shape->D;
  const int64_t Hkv = shape->Hkv == 0 ? H : shape->Hkv;
  if (T < 0 || B < 0 || H < 0 || Hkv < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative size");
  if (D <= 0) return api_fail(JVP_ERR_INVALID_ARG, "D must be positive");
  if (D > 128) return api_fail(JVP_ERR_UNSUPPORTED, "D > 128 is not supported");
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  if (!in_strides || !out_strides) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  if (!std::isfinite(scale)) return api_fail(JVP_ERR_INVALID_ARG, "scale is not finite");
  if (causal != 0 && causal != 1) return api_fail(JVP_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (H > 0 && H % Hkv != 0)
    return api_fail(JVP_ERR_INVALID_ARG, "H must be a multiple of Hkv (grouped-query attention)");
  // the largest grid: one block per (query head, 1-row sequence or tile)
  if (T > kMax || B > kMax || H > kMax || T + B > kMaxRows || (H > 0 && T + B > kMax / H))
    return api_fail(JVP_ERR_UNSUPPORTED, "problem too large for one launch");
  for (int i = 0; i < 4; ++i) {
    const jvp_status_t st = check_strides(i < 3 ? in_strides[i] : *out_strides,
                                          "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
  }
  if ((T > 1 && out_strides->n == 0) || (H > 1 && out_strides->h == 0))
    return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  if (T == 0 || B == 0 || H == 0) return api_ok();
  if (!q || !k || !v || !o || !cu_seqlens)
    return api_fail(JVP_ERR_INVALID_ARG, "q, k, v, o or cu_seqlens is NULL");
  const int64_t e = elem_bytes(dtype);
  if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(o, e))
    return api_fail(JVP_ERR_ALIGNMENT, "a tensor is not aligned to its element size");
  if (!aligned_to(lse, 4) || !aligned_to(cu_seqlens, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "lse or cu_seqlens not 4-byte aligned");
  int sms = 0;
  unsigned int* status = nullptr;
  const jvp_status_t st = api_device(&sms, &status);
  if (st != JVP_OK) return st;

  PackedParams p{};
  p.T = static_cast<int>(T), p.B = static_cast<int>(B), p.H = static_cast<int>(H);
  p.Hkv = static_cast<int>(Hkv), p.D = static_cast<int>(D), p.group = static_cast<int>(H / Hkv);
  p.causal = causal;
  p.scale = scale, p.scale_log2 = scale * 1.4426950408889634f;
  p.cu = cu_seqlens;
  p.q = q, p.k = k, p.v = v, p.o = o, p.lse = lse, p.status = status;
  p.sq = used(in_strides[0], 0, H, T), p.sk = used(in_strides[1], 0, Hkv, T);
  p.sv = used(in_strides[2], 0, Hkv, T), p.so = used(*out_strides, 0, H, T);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool tc = e == 2 && D % 8 == 0 && p.group <= kPackedTileRows && scale != 0.f &&
            aligned_to(o, 16) && multiple(p.so, 8);
  PackedMaps maps;
  if (tc) {
    // Q, O: boxes of `tok` tokens times a key/value head's query heads; K, V: key
    // tiles of one head.  (D < 64 or 128: columns past D are zero-filled.)
    p.tok = kPackedTileRows / p.group;
    tc = encode_packed(&maps.q, dtype, q, D, H, p.sq.h, T, p.sq.n, p.group, p.tok) &&
         encode_packed(&maps.o, dtype, o, D, H, p.so.h, T, p.so.n, p.group, p.tok) &&
         encode_packed(&maps.k, dtype, k, D, T, p.sk.n, Hkv, p.sk.h, kPackedBlockN, 1) &&
         encode_packed(&maps.v, dtype, v, D, T, p.sv.n, Hkv, p.sv.h, kPackedBlockN, 1);
  }
  cudaError_t err;
  if (tc) {
    // Two query tiles per CTA share each K/V tile and keep the tensor core
    // busy; one tile per CTA and two CTAs per SM overlap the ends of short
    // prompts instead.  Measured by average length (16384 tokens, 16/4 heads,
    // D = 128, one against two tiles): 128 52.4 / 58.4 us, 512 79.2 / 80.6
    // (causal 67.9 / 68.5), 1024 122.6 / 120.6 (90.5 / 88.2), 4096 382 / 357
    // (222 / 204); 16/16 heads D = 64: 128 62.2 / 85.2, 512 65.2 / 67.8
    // (57.5 / 67.8), 1024 101.8 / 96.8 (75.8 / 82.5), 4096 330 / 277 (182 / 178).
    // At D > 64 also where the pairs would leave SMs idle (one prompt, one
    // against two: 2048 tokens, 8/8 heads, 64 pairs 26.2 / 28.7 us, causal 26.9
    // / 29.5; 2142 tokens, 12/4 heads, 104 pairs, D = 80, 35.8 / 30.9, causal
    // 28.8 / 30.9; 4096 tokens, 4/4 heads of 64, 64 pairs 40.1 / 39.4).
    const int64_t pairs = (T + 2 * p.tok - 1) / (2 * p.tok) * Hkv;
    p.query_tiles = T <= (causal ? 768 : 512) * B || (D > 64 && pairs <= (causal ? sms : sms / 2))
                        ? 1
                        : 2;
    // >= sum of ceil(length / tokens of a CTA)
    p.tiles = static_cast<int>(T / (p.query_tiles * p.tok) + B);
    // as many key/value heads side by side as keep their rows within 32 MB of L2
    p.head_group = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(Hkv, (32ll << 20) / std::max<int64_t>(1, T * D * 2 * e))));
    if (scale < 0.f) {  // negated score products, |scale|
      p.neg_scores = 1;
      p.scale = -p.scale, p.scale_log2 = -p.scale_log2;
    }
    err = launch_packed_tc(static_cast<DType>(dtype), D <= 64 ? 64 : 128, maps, p, s);
  } else {
    p.tiles = static_cast<int>(T / kPackedSimtRows + B);
    p.vec = e == 4 && D % 4 == 0 && aligned_to(q, 16) && aligned_to(k, 16) && aligned_to(v, 16) &&
            multiple(p.sq, 4) && multiple(p.sk, 4) && multiple(p.sv, 4);
    err = launch_packed_simt(static_cast<DType>(dtype), p, s);
  }
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(tc ? 1 : 2);
  return api_ok();
}

jvp_status_t jvp_attn_cache_write(const jvp_cache_t* cache, jvp_dtype_t dtype, int64_t T,
                                  const void* k, const void* v, const jvp_strides_t* in_strides,
                                  const int32_t* block_table, const int32_t* start_pos,
                                  const int32_t* cu_seqlens, void* k_cache, void* v_cache,
                                  uint8_t* k_scale, uint8_t* v_scale, void* stream) {
  return jvp::cache_rows(true, cache, dtype, T, k, v, in_strides, block_table, start_pos,
                         cu_seqlens, k_cache, v_cache, k_scale, v_scale, stream);
}

jvp_status_t jvp_attn_cache_read(const jvp_cache_t* cache, jvp_dtype_t dtype, int64_t T,
                                 const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                                 const uint8_t* v_scale, const int32_t* block_table,
                                 const int32_t* start_pos, const int32_t* cu_seqlens, void* k,
                                 void* v, const jvp_strides_t* out_strides, void* stream) {
  return jvp::cache_rows(false, cache, dtype, T, k, v, out_strides, block_table, start_pos,
                         cu_seqlens, k_cache, v_cache, k_scale, v_scale, stream);
}

size_t jvp_attn_decode_workspace_size(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype) {
  if (jvp::check_decode(cache, H, dtype) != JVP_OK || H == 0 || cache->B == 0) return 0;
  int sms = 0;
  unsigned int* status = nullptr;
  if (jvp::api_device(&sms, &status) != JVP_OK) return 0;
  // enough for either path (which one runs depends on the pointers too)
  return std::max(jvp::plan_decode(cache, H, true, sms, 0, 0).bytes,
                  jvp::plan_decode(cache, H, false, sms, 0, 0).bytes);
}

jvp_status_t jvp_attn_decode(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype, const void* q,
                             const jvp_strides_t* q_strides, const void* k_cache,
                             const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                             const int32_t* block_table, const int32_t* seq_lens, float scale,
                             void* o, const jvp_strides_t* o_strides, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return jvp::decode(cache, H, dtype, q, q_strides, k_cache, v_cache, k_scale, v_scale, block_table,
                     seq_lens, 0, 0, scale, o, o_strides, lse, workspace, workspace_bytes, stream);
}

jvp_status_t jvp_attn_decode_window(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype,
                                    const void* q, const jvp_strides_t* q_strides,
                                    const void* k_cache, const void* v_cache,
                                    const uint8_t* k_scale, const uint8_t* v_scale,
                                    const int32_t* block_table, const int32_t* seq_lens,
                                    int64_t window, int64_t sinks, float scale, void* o,
                                    const jvp_strides_t* o_strides, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (const char* why = jvp::bad_window(window, sinks)) {
    jvp::api_set_path(0);
    return jvp::api_fail(JVP_ERR_INVALID_ARG, why);
  }
  return jvp::decode(cache, H, dtype, q, q_strides, k_cache, v_cache, k_scale, v_scale, block_table,
                     seq_lens, std::min(window, jvp::kMax), std::min(sinks, jvp::kMax), scale, o,
                     o_strides, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
