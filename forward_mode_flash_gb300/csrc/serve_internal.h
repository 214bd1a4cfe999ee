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

cudaError_t launch_decode(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
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
