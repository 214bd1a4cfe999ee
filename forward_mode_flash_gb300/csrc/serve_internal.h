// serve_internal.h -- launch descriptions of the packed-prompt attention, the
// paged key-value cache and the single-token attention over it (not part of
// the public ABI).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "jvp_attn.h"
#include "jvp_internal.h"

namespace jvp {

// Bit of the device status word: a page index, length or offset read on the
// device was out of range (the rows it would have reached were skipped).
constexpr unsigned kStatusIndex = 4u;

// The caller's cache: key rows [pages, Hkv, page_size, D] (strides b, h, n in
// elements), value rows likewise, one scale byte per (page, head, row) of an
// e4m3 cache, and the sequences' pages.
struct PagedCache {
  int pages, Hkv, page_size, D;
  int page_shift;  // log2(page_size) where that is a whole number, else -1
  int B, max_pages;
  long long table_stride;
  const int* table;
  void *k, *v;
  Strides sk, sv;
  uint8_t *k_scale, *v_scale;
  unsigned int* status;
};

struct CacheRowsParams {
  PagedCache c;
  long long T;      // rows of the packed tensors
  const int* cu;    // [B + 1], or nullptr: row r belongs to sequence r
  const int* start; // [B] position of each sequence's first row, or nullptr: 0
  const void *k, *v;  // rows to write (or, reading, outputs)
  Strides srk, srv;
  int vec;          // 16-byte pieces per lane that alignment and D allow: 0, 1 or 2 (e4m3: 0
                    // where the scales of a page are more than 2^31 - 1)
};
// Writes packed rows into the cache / reads them back.  dt: type of the packed
// rows; e4m3: the cache holds codes and scales, else entries of type dt.
cudaError_t launch_cache_write(DType dt, bool e4m3, const CacheRowsParams& p, cudaStream_t stream);
cudaError_t launch_cache_read(DType dt, bool e4m3, const CacheRowsParams& p, cudaStream_t stream);

// Norms per head and rotation by position.
struct RopeParams {
  int D, rot;           // rot: rotated columns (even, at most D; 0: none)
  int interleaved;      // pairs are neighbours, else half a rotation apart
  int table_rows;
  const float* table;   // [table_rows][rot]: cosines, then sines, of the pairs
  const void *wq, *wk;  // [D] each, or nullptr both: no norms
  int weight_type;      // DType of the weights
  float eps, inv_d;
  unsigned int* status;
};
// Dense rows [B, H, N, D].  Tensors by index: queries and keys (0, 1), their
// tangents (2, 3), backward also cotangents (4, 5) and those of the tangents (6, 7).
struct RopeDense {
  RopeParams r;
  long long tokens;  // B * N
  int N, H, Hkv;
  const int* positions;  // [B, N], or nullptr: 0 .. N - 1
  long long positions_stride;
  const void* x[8];
  Strides in[8];
  void* y[4];
  Strides out[4];
  int back;          // without norms: rotate back
  float* ws;         // [blocks][2][D] sums of the weights' gradients
  float *gwq, *gwk;  // [D]
  long long units;   // set by the launch: warps' work
  int heads_per_unit, head_chunks;
};
constexpr int rope_blocks_per_sm() { return 4; }  // at most, where blocks leave sums
// vec: 16-byte aligned rows of whole pieces; bwd: the gradients.
cudaError_t launch_norm_rope(DType dt, bool vec, bool bwd, RopeDense d, int num_sms,
                             cudaStream_t stream);

struct AppendParams {
  RopeParams r;
  PagedCache c;
  long long T;
  int H;
  const int *cu, *start;
  const void* x[3];  // q, k, v
  Strides in[3];
  void* q_out;
  Strides sq_out;
  long long units;
  int heads_per_unit, head_chunks;
};
cudaError_t launch_cache_append(DType dt, bool e4m3, bool vec, AppendParams a, int num_sms,
                                cudaStream_t stream);

struct DecodeParams {
  PagedCache c;
  int H, group;        // query heads, and query heads per key/value head
  int head_blocks;     // blocks of heads_per_block query heads per key/value head
  int grid;            // CTAs of the attention kernel (the partial states' slots)
  int direct;          // 1: CTA i takes segment i whole; no join
  const int* lens;     // [B] keys of each sequence
  const void* q;
  Strides sq;          // b, h
  void* o;
  Strides so;
  float* lse;          // [B, H] or nullptr
  float scale_log2;    // logit scale * log2(e)
  float* ws_lse;       // [grid][2][heads_per_block]
  float* ws_o;         // [grid][2][heads_per_block][64 or 128]
  int2* ws_cta;        // [B][Hkv][head_blocks] first and last CTA of a segment
  int o_vec;           // output rows are 16-byte aligned
  int window, sinks;   // (launch_decode_window) keys j >= lens[b] - window or j < sinks are visible
};

// Which kernel a call takes: tensor cores (16-bit queries, 16-byte aligned
// rows, D a multiple of 8, of 16 for an e4m3 cache) or CUDA cores.
// Query heads per CTA: 8 or 16 of a key/value head's group on the tensor
// cores, 1 (ungrouped heads) or 4 on the CUDA cores.
inline int decode_heads_per_block(bool tc, int group) {
  if (tc) return group > 8 ? 16 : 8;
  return group > 1 ? 4 : 1;
}
// Tensor cores: keys of a warp's group of rows (K and V rows of 8 KB at most)
// and groups in a warp's ring; four warps' groups are the split's tile.
// (e4m3, 64 sequences, 16/2 heads of 128: 57.1 us as here; three stages at two
// CTAs per SM 64.4; groups of 16 keys in three stages at three CTAs 69.2, in two
// stages at four CTAs 64.2.)
constexpr int decode_warp_keys(int D, bool e4m3) { return D > 64 && !e4m3 ? 16 : 32; }
constexpr int decode_stages(bool e4m3) { return e4m3 ? 2 : 3; }
constexpr int kDecodeSimtTile = 64;
constexpr int decode_simt_ctas_per_sm(int heads) { return heads > 1 ? 3 : 4; }
constexpr int decode_tile(bool tc, int D, bool e4m3) {
  return tc ? 4 * decode_warp_keys(D, e4m3) : kDecodeSimtTile;
}
// CTAs per SM that the split is made for: one resident wave (shared memory of
// the rings, 64 or 96 KB; registers, 168 a thread at three CTAs of 128).
constexpr int decode_ctas_per_sm(int D, int head_groups, bool e4m3) {
  return !e4m3 || (D > 64 && head_groups > 1) ? 2 : 3;
}
// Where no sequence can have more tiles than this, a CTA takes a whole segment
// and nothing is joined.
constexpr int kDecodeDirectTiles = 4;
// The same on the tensor cores where a window leaves every sequence so few tiles: more, since
// a split and its join cost 2 us and more, and with a segment for every SM as many as a CTA
// reads while the others' parts would be joined.  A tile is 64 keys of 16 bits at D > 64, else
// 128.  Direct against split, us in a graph, D = 128 (96 is alike), by window:
//   few segments     8 x 16/4 heads, bf16   300 7.8 / 8.1    500 9.8 / 9.2
//                    8 x 16/1 heads, bf16   200 8.1 / 8.4    300 9.6 / 8.7
//                    8 x 16/4 heads, e4m3   300 8.2 / 8.2    400 9.2 / 8.6
//                    8 x 16/1 heads, e4m3   300 10.5 / 9.8   400 11.8 / 10.0
//   one for each SM  40 x 16/4 heads, bf16  700 13.7 / 16.0  1000 18.0 / 17.4  2000 32 / 33
//                    160 x 16/1 heads, bf16 700 17.6 / 25.2  1000 22.8 / 27.1  2000 40 / 42
//                    40 x 16/4 heads, e4m3  1000 16.4 / 17.2 1500 21.2 / 19.7  2000 27 / 22
//                    160 x 16/1 heads, e4m3 1000 21.1 / 31.4 1500 27.7 / 33.6  2000 34 / 36
//   many             200 x 16/4 heads, bf16 700 52 / 57      1000 69 / 74
//                    200 x 16/4 heads, e4m3 1000 44 / 52     2000 76 / 81
// and D = 64: 8 x 16/4 heads, bf16, 600 7.5 / 8.0, e4m3 500 8.0 / 8.6; 8 x 16/1 heads, bf16, 500
// 8.3 / 8.1, e4m3 300 9.1 / 8.9; 40 x 16/4 heads, bf16, 700 9.2 / 12.7, e4m3 700 10.8 / 13.5.
constexpr int decode_window_direct(int D, bool e4m3, int heads_per_block, bool enough) {
  if (enough) return D <= 64 ? 6 : e4m3 ? 9 : 18;  // (some 750 and 1100 keys)
  return 6 - (e4m3 ? 1 : 0) - (heads_per_block > 8 ? 1 : 0);
}

cudaError_t launch_decode(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
                          cudaStream_t stream);
cudaError_t launch_decode_window(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
                                 cudaStream_t stream);

struct PackedParams {
  int T, B, H, Hkv, D, group;
  int causal;
  int tok;             // query tokens of one 128-row tile (tensor cores): 128 / group
  int tiles;           // upper bound of the blocks a key/value head needs
  int query_tiles;     // tensor cores: query tiles of a CTA (1 or 2)
  int head_group;      // tensor cores: key/value heads scheduled together
  float scale, scale_log2;
  int neg_scores;      // scale < 0: the score products are formed negated, |scale| applied
  const int* cu;
  const void *q, *k, *v;
  Strides sq, sk, sv;  // h, n
  void* o;
  Strides so;
  float* lse;          // [H, T] or nullptr
  int vec;             // CUDA cores: fp32 input rows are 16-byte aligned, D % 4 == 0
  unsigned int* status;
};
struct PackedMaps {
  CUtensorMap q, k, v, o;
};
// Tensor-core kernel (fp16 / bf16, D a multiple of 8 up to 128, group <= 128).
cudaError_t launch_packed_tc(DType dt, int kernel_d, const PackedMaps& maps, const PackedParams& p,
                             cudaStream_t stream);
constexpr int kPackedTileRows = 128;  // rows of a query tile; a CTA has two
constexpr int kPackedBlockN = 128;    // keys per tile
// CUDA-core kernel (any type, any D up to 128).
cudaError_t launch_packed_simt(DType dt, const PackedParams& p, cudaStream_t stream);
constexpr int kPackedSimtRows = 32;

// Attention of chunks of new tokens over a paged cache.  Token i of a sequence's
// len has position lens[b] - len + i and sees the keys at positions up to its own
// (with a window: of these the last `window`, and the first `sinks`).
struct ChunkParams {
  PagedCache c;
  int T, H, group;
  int tok;           // query tokens of a tile of rows
  int query_tiles;   // tensor cores: tiles of rows of a CTA (1 or 2)
  int head_blocks;   // CUDA cores: blocks of `group_rows` query heads per key/value head
  int group_rows;    // query heads of a tile's rows
  int window, sinks; // window 0: none
  float scale_log2;
  int neg_scores;    // scale < 0: the score products are formed negated, |scale| applied
  const int *cu, *lens;
  const void* q;
  Strides sq;
  void* o;
  Strides so;
  float* lse;        // [H, T] or nullptr
  int heads;         // key/value heads times head_blocks: items of a tile of tokens
  // The division among CTAs (chunk.cuh)
  int grid;
  int cut;           // 0: items are not cut (their key tiles are few)
  int4* ws_item;     // [grid] the item that a CTA begins and others end: CTAs, first row,
                     // tokens, head (CTAs 0: none)
  float* ws_o;       // [grid][2][rows of an item][64 or 128] normalised partial outputs
  float* ws_lse;     // [grid][2][rows of an item], log2 units
  int box_rows;      // tensor cores: keys of a copied box, a divisor of 128 and the page size
  int vec;           // CUDA cores: rows of whole pieces of four elements, aligned to these
};
struct ChunkMaps {
  CUtensorMap q, o, k, v;
};
constexpr int kChunkTile = 128, kChunkSimtTile = 64, kChunkSimtRows = 32;  // keys per tile, rows
// Cost of an item beside its key tiles, in tiles, the least cost for a CTA, and the fewest
// tiles of a part of a cut item.  A tile of the CUDA cores' kernel takes 3 us, so one is
// worth a CTA: 1, 3, 1 against the other's 4, 9, 4, us, fp32, 8/2 heads: 4 chunks of 150
// tokens over 512 positions 36 / 57, a token over 5120 36 / 54, 100 over 1024 66 / 85, 2 of
// 2000 over 4096 796 / 825.  (3, 8, 3 and 4, 8, 2 on the tensor cores: within 3%.)
struct ChunkCost {
  int start, least, snap;
};
constexpr ChunkCost chunk_cost(int tile) {
  return tile == kChunkTile ? ChunkCost{4, 9, 4} : ChunkCost{1, 3, 1};
}
// source of the key tiles: boxes of parts of pages by TMA, rows gathered by threads,
// e4m3 rows gathered and converted, or copied by TMA and converted
enum ChunkSource { kChunkBoxes, kChunkRows, kChunkE4M3, kChunkStaged };
cudaError_t launch_chunk_tc(DType dt, int kernel_d, ChunkSource source, const ChunkMaps& maps,
                            const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_simt(DType dt, bool e4m3, const ChunkParams& p, cudaStream_t stream);
// Joins the pieces of split items (rows: of an item; kernel_d: 64 or 128).
cudaError_t launch_chunk_join(DType dt, int kernel_d, int rows, const ChunkParams& p,
                              cudaStream_t stream);
// Launches a kernel that may be placed while the one before it on the stream runs,
// and waits for it by itself (griddepcontrol.wait).
template <typename... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem,
                             cudaStream_t stream, const P&... params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device.
// Once per kernel and device (the call costs 2 us of an eager call's host time;
// making it twice is harmless).
template <auto KERN>
cudaError_t allow_shared_memory(int bytes) {
  static std::atomic<unsigned long long> done{0};
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) & (1ull << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// What the entry points of the other translation unit share with jvp_attn_api.cu.
jvp_status_t api_fail(jvp_status_t s, const char* msg);
jvp_status_t api_cuda_fail(cudaError_t e);
jvp_status_t api_ok();
void api_set_path(int path);
// Current device: JVP_OK with its SM count and status word, or the error.
jvp_status_t api_device(int* num_sms, unsigned int** status);
// cuTensorMapEncodeTiled, or nullptr.
void* api_tensor_map_encoder();

}  // namespace jvp
