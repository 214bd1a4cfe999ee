// chunk_api.cu -- entry point of the attention of chunks of new tokens over a
// paged cache: argument checks, path selection and launch descriptions.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "serve_checks.h"

namespace jvp {
namespace {

// How a call's work is divided (see chunk.cuh), and its workspace.
struct ChunkPlan {
  int tok = 0, query_tiles = 1, head_blocks = 1, group_rows = 1;
  int rows = 0;  // of an item
  int64_t heads = 0;
  int tile = 0, grid = 0, cut = 0;
  size_t bytes = 0, at_lse = 0, at_o = 0;  // workspace: items, ...
};
// Query tiles of a CTA (0 stands for the CUDA cores' kernel): two share each K/V tile,
// unless a chunk fills no more than one on average, when one per CTA and two CTAs per SM
// hide each other's beginnings and ends.  One against two, us, pages of 16: D = 128, 8/8
// heads, 64 chunks of 128 tokens over 2048 positions 123 / 132, 32 of 256 111 / 98, 8 of
// 1024 over 8192 290 / 216; 16/2 heads, 32 of 16 over 5120 60 / 58; D = 64, 8/8 heads, 32
// of 16 85 / 110, 64 of 128 84 / 103, 4 of 4096 with a window of 1024 111 / 100.  Gathered
// rows leave room for one CTA per SM.
int chunk_query_tiles(const jvp_cache_t* c, int64_t H, int64_t T, bool boxes) {
  return boxes && T * (H / c->Hkv) <= kPackedTileRows * c->B ? 1 : 2;
}
ChunkPlan plan_chunk(const jvp_cache_t* c, int64_t H, int64_t T, int query_tiles, int num_sms,
                     int64_t window, int64_t sinks) {
  ChunkPlan d;
  const int64_t group = H / c->Hkv;
  int ctas;  // resident
  if (query_tiles > 0) {
    d.query_tiles = query_tiles;
    d.group_rows = static_cast<int>(group);
    d.tok = static_cast<int>(kPackedTileRows / group);
    d.rows = d.query_tiles * kPackedTileRows;
    d.tile = kChunkTile;
    ctas = num_sms * (3 - d.query_tiles);
  } else {
    d.group_rows = static_cast<int>(std::min<int64_t>(group, kChunkSimtRows));
    d.head_blocks = static_cast<int>((group + d.group_rows - 1) / d.group_rows);
    d.tok = kChunkSimtRows / d.group_rows;
    d.rows = kChunkSimtRows;
    d.tile = kChunkSimtTile;
    ctas = num_sms * (c->D > 64 ? 2 : 3);
  }
  d.heads = c->Hkv * d.head_blocks;
  const int64_t step = static_cast<int64_t>(d.tok) * d.query_tiles;
  const int64_t items = T / step + std::min(c->B, T);  // >= sum of ceil(len / step)
  int64_t tiles = (c->max_pages * c->page_size + d.tile - 1) / d.tile;
  if (window > 0)  // the window's keys of `step` tokens begin anywhere in a tile
    tiles = std::min(tiles, (window + step - 2 + d.tile - 1) / d.tile + 1 +
                                (sinks + d.tile - 1) / d.tile);
  tiles = std::max<int64_t>(tiles, 1);
  // (items of so few tiles are not worth a join; items * heads <= 2^31 - 1, checked by the
  // caller, tiles < 2^31)
  const ChunkCost cost = chunk_cost(d.tile);
  d.cut = tiles >= 2 * cost.snap ? 1 : 0;
  d.grid = static_cast<int>(
      std::min<int64_t>(ctas, items * d.heads * (tiles + cost.start) / cost.least + 1));
  auto place = [&](size_t* at, size_t bytes) {
    *at = d.bytes;
    d.bytes += (bytes + 255) & ~static_cast<size_t>(255);
  };
  const size_t grid = static_cast<size_t>(d.grid);
  size_t at_item;
  place(&at_item, grid * 16);
  if (d.cut) {
    const size_t rows = 2 * grid * d.rows;
    place(&d.at_lse, rows * 4);
    place(&d.at_o, rows * (c->D > 64 ? 128 : 64) * 4);
  }
  return d;
}

jvp_status_t check_chunk(const jvp_cache_t* c, int64_t H, int dtype, int64_t T) {
  const jvp_status_t st = check_cache(c, false);
  if (st != JVP_OK) return st;
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  if (c->dtype != JVP_E4M3 && c->dtype != dtype)
    return api_fail(JVP_ERR_INVALID_ARG, "q must have the cache's dtype (or the cache e4m3)");
  if (T < 0 || H < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative T or H");
  if (c->Hkv == 0 ? H > 0 : H % c->Hkv != 0)
    return api_fail(JVP_ERR_INVALID_ARG, "H must be a multiple of Hkv (grouped-query attention)");
  // the largest grid: one block per (query head, 1-row sequence or tile)
  if (T > kMax || H > kMax || T + c->B > kMaxRows || (H > 0 && T + c->B > kMax / 4 / H))
    return api_fail(JVP_ERR_UNSUPPORTED, "problem too large for one launch");
  return JVP_OK;
}

// Map of a cache [pages, Hkv, page_size, D], boxes of `rows` rows of one head: 64 columns
// of 16 bits with a swizzle of 128 bytes, or all columns (64 or 128) of 8 bits.
bool encode_cache(CUtensorMap* map, int dt, const void* ptr, const PagedCache& c, const Strides& s,
                  int rows) {
  const bool codes = dt == JVP_E4M3;
  const cuuint64_t e = codes ? 1 : 2;
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(api_tensor_map_encoder());
  if (!enc || !aligned_to(ptr, 16)) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                        static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.pages)};
  // a size-1 dimension's stride is never used; give it a well-formed value
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.page_size > 1 ? s.n : c.D) * e,
                           static_cast<cuuint64_t>(c.Hkv > 1 ? s.h : c.D) * e,
                           static_cast<cuuint64_t>(c.pages > 1 ? s.b : c.D) * e};
  for (auto x : strides)
    if (x == 0 || x % 16 != 0 || x >= (1ull << 40)) return false;
  cuuint32_t box[4] = {codes && c.D > 64 ? 128u : 64u, static_cast<cuuint32_t>(rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map,
             codes            ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : dt == JVP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             4, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace jvp

extern "C" {

size_t jvp_attn_chunk_workspace_size(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype,
                                     int64_t T) {
  using namespace jvp;
  if (check_chunk(cache, H, dtype, T) != JVP_OK || H == 0 || T == 0 || cache->B == 0) return 0;
  int sms = 0;
  unsigned int* status = nullptr;
  if (api_device(&sms, &status) != JVP_OK) return 0;
  // enough for each kernel (which one runs depends on the pointers too) and any window
  size_t most = 0;
  for (int tiles = 0; tiles <= (H / cache->Hkv <= kPackedTileRows ? 2 : 0); ++tiles)
    most = std::max(most, plan_chunk(cache, H, T, tiles, sms, 0, 0).bytes);
  return most;
}

jvp_status_t jvp_attn_chunk(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype, int64_t T,
                            const void* q, const jvp_strides_t* q_strides, const void* k_cache,
                            const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                            const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* cu_seqlens, int64_t window, int64_t sinks, float scale,
                            void* o, const jvp_strides_t* o_strides, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  using namespace jvp;
  api_set_path(0);
  jvp_status_t st = check_chunk(cache, H, dtype, T);
  if (st != JVP_OK) return st;
  if (!std::isfinite(scale)) return api_fail(JVP_ERR_INVALID_ARG, "scale is not finite");
  if (window < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative window");
  if (sinks < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative number of sinks");
  if (!q_strides || !o_strides) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  for (const jvp_strides_t* s : {q_strides, o_strides}) {
    st = check_strides(*s, "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
  }
  if ((T > 1 && o_strides->n == 0) || (H > 1 && o_strides->h == 0))
    return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  const int64_t B = cache->B, D = cache->D;
  if (B == 0 || H == 0 || T == 0) return api_ok();
  if (!q || !o || !seq_lens || !cu_seqlens)
    return api_fail(JVP_ERR_INVALID_ARG, "q, o, seq_lens or cu_seqlens is NULL");
  const int64_t e = elem_bytes(dtype), ce = elem_bytes(cache->dtype);
  if (!aligned_to(q, e) || !aligned_to(o, e))
    return api_fail(JVP_ERR_ALIGNMENT, "q or o not aligned to its element size");
  if (!aligned_to(lse, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_seqlens, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "lse, seq_lens or cu_seqlens not 4-byte aligned");
  st = check_cache_ptrs(cache, k_cache, v_cache, k_scale, v_scale, block_table);
  if (st != JVP_OK) return st;
  int sms = 0;
  unsigned int* status = nullptr;
  st = api_device(&sms, &status);
  if (st != JVP_OK) return st;

  ChunkParams p{};
  p.c = describe(cache, k_cache, v_cache, k_scale, v_scale, block_table, status);
  p.T = static_cast<int>(T), p.H = static_cast<int>(H), p.group = static_cast<int>(H / cache->Hkv);
  // (a window that is wider than any sequence hides nothing)
  const int64_t most = cache->max_pages * cache->page_size;
  p.window = window >= most ? 0 : static_cast<int>(window);
  p.sinks = p.window > 0 ? static_cast<int>(std::min(sinks, most)) : 0;
  p.cu = cu_seqlens, p.lens = seq_lens;
  p.q = q, p.sq = used(*q_strides, 0, H, T);
  p.o = o, p.so = used(*o_strides, 0, H, T);
  p.lse = lse;
  p.scale_log2 = scale * 1.4426950408889634f;
  const bool e4m3 = cache->dtype == JVP_E4M3;
  bool tc = e == 2 && D % 8 == 0 && p.group <= kPackedTileRows && scale != 0.f &&
            aligned_to(o, 16) && multiple(p.so, 8) && aligned_to(k_cache, 8 * ce) &&
            aligned_to(v_cache, 8 * ce) && multiple(p.c.sk, 8) && multiple(p.c.sv, 8);
  ChunkSource source = e4m3 ? kChunkE4M3 : kChunkRows;
  ChunkMaps maps{};
  if (tc) {
    const int tok = kPackedTileRows / p.group;
    tc = encode_packed(&maps.q, dtype, q, D, H, p.sq.h, T, p.sq.n, p.group, tok) &&
         encode_packed(&maps.o, dtype, o, D, H, p.so.h, T, p.so.n, p.group, tok);
  }
  if (tc && cache->page_size % 8 == 0) {  // (of e4m3 rows, half a tile at most)
    int rows = 8;
    while (rows < kChunkTile / (e4m3 ? 2 : 1) && cache->page_size % (2 * rows) == 0) rows *= 2;
    if (encode_cache(&maps.k, cache->dtype, k_cache, p.c, p.c.sk, rows) &&
        encode_cache(&maps.v, cache->dtype, v_cache, p.c, p.c.sv, rows)) {
      p.box_rows = rows;
      source = e4m3 ? kChunkStaged : kChunkBoxes;
    }
  }
  const int query_tiles = tc ? chunk_query_tiles(cache, H, T, source == kChunkBoxes) : 0;
  const ChunkPlan d = plan_chunk(cache, H, T, query_tiles, sms, p.window, p.sinks);
  if (!workspace || workspace_bytes < d.bytes)
    return api_fail(JVP_ERR_WORKSPACE,
                    "workspace is NULL or smaller than jvp_attn_chunk_workspace_size()");
  if (!aligned_to(workspace, 16)) return api_fail(JVP_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  p.tok = d.tok, p.query_tiles = d.query_tiles;
  p.head_blocks = d.head_blocks, p.group_rows = d.group_rows;
  p.heads = static_cast<int>(d.heads);
  p.grid = d.grid, p.cut = d.cut;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ws_item = reinterpret_cast<int4*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + d.at_lse);
  p.ws_o = reinterpret_cast<float*>(ws + d.at_o);
  const int kernel_d = D <= 64 ? 64 : 128;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tc && scale < 0.f) p.neg_scores = 1, p.scale_log2 = -p.scale_log2;
  if (!tc)
    p.vec = D % 4 == 0 && aligned_to(k_cache, 4 * ce) && aligned_to(v_cache, 4 * ce) &&
            multiple(p.c.sk, 4) && multiple(p.c.sv, 4);
  cudaError_t err = tc ? launch_chunk_tc(static_cast<DType>(dtype), kernel_d, source, maps, p, s)
                       : launch_chunk_simt(static_cast<DType>(dtype), e4m3, p, s);
  if (err == cudaSuccess && d.cut)
    err = launch_chunk_join(static_cast<DType>(dtype), kernel_d, d.rows, p, s);
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(tc ? 1 : 2);
  return api_ok();
}

}  // extern "C"
