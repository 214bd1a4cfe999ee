// chunk_join.cu -- joins the pieces of cut items of the attention of chunks: per
// row, partial outputs weighted by their log-sum-exps, in the order of the keys.
//
// A warp takes a row at a time; the blocks share the rows of the slots that the
// attention kernel says are in use (none where nothing was cut).  The kernel may be
// placed while that one runs, and waits for its end.
#include <cmath>

#include "debug_checks.cuh"
#include "rows.cuh"
#include "serve_internal.h"

namespace jvp {
namespace {

constexpr int kJoinWarps = 8;

template <typename T, int DPAD>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const ChunkParams p, int rows) {
  constexpr int C = DPAD / 32;  // columns of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_rows = rows / p.query_tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int slots = *static_cast<volatile int*>(p.ws_count);
  const long long units = static_cast<long long>(slots) * (rows / kJoinWarps);
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int slot = static_cast<int>(u / (rows / kJoinWarps));
    const int row = static_cast<int>(u % (rows / kJoinWarps)) * kJoinWarps + warp;
    const int4 item = p.ws_item[slot];  // pieces, first row, tokens, head
    if (item.x == 0) continue;
    const int x = row / tile_rows, r = row - x * tile_rows;
    const int rt = r / p.group_rows, rh = r - rt * p.group_rows;
    const int token = x * p.tok + rt;
    const int hk = item.w / p.head_blocks;
    const int in_group = (item.w - hk * p.head_blocks) * p.group_rows + rh;
    if (rt >= p.tok || token >= item.z || in_group >= p.group) continue;
    float M = -INFINITY, L = 0.f, acc[C];
#pragma unroll
    for (int k = 0; k < C; ++k) acc[k] = 0.f;
    constexpr int U = 4;  // pieces in flight
    for (int i = 0; i < item.x; i += U) {
      float y[U], v[U][C];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        y[k] = -INFINITY;
#pragma unroll
        for (int d = 0; d < C; ++d) v[k][d] = 0.f;
        const long long at = (static_cast<long long>(slot) + static_cast<long long>(i + k) * p.heads) *
                                 rows + row;
        if (i + k >= item.x ||
            !JVP_CHECK(at < static_cast<long long>(p.slots) * rows, p.c.status, kChkGlobalRow))
          continue;
        y[k] = p.ws_lse[at];
        if constexpr (C == 4) {
          const float4 w = *reinterpret_cast<const float4*>(p.ws_o + at * DPAD + lane * C);
          v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
        } else {
          const float2 w = *reinterpret_cast<const float2*>(p.ws_o + at * DPAD + lane * C);
          v[k][0] = w.x, v[k][1] = w.y;
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float m = fmaxf(M, y[k]), mu = m == -INFINITY ? 0.f : m;
        const float a = exp2f(M - mu), w = exp2f(y[k] - mu);
        M = m;
        L = L * a + w;
#pragma unroll
        for (int d = 0; d < C; ++d) acc[d] = fmaf(w, v[k][d], acc[d] * a);
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int h = hk * p.group + in_group;
    const long long t = static_cast<long long>(item.y) + token;
    if (!JVP_CHECK(t < p.T && h < p.H, p.c.status, kChkGlobalRow)) continue;
    T* dst = static_cast<T*>(p.o) + t * p.so.n + h * p.so.h;
#pragma unroll
    for (int d = 0; d < C; ++d)
      if (lane * C + d < p.c.D) dst[lane * C + d] = Rows<T>::put(acc[d] * inv);
    if (lane == 0 && p.lse)
      p.lse[h * static_cast<long long>(p.T) + t] =
          L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

template <typename T>
cudaError_t launch_typed(int kernel_d, int rows, const ChunkParams& p, int num_sms,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const long long units = static_cast<long long>(p.slots) * (rows / kJoinWarps);
  const long long most = 8ll * num_sms;
  cfg.gridDim = dim3(static_cast<unsigned>(units < most ? units : most));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return kernel_d > 64 ? cudaLaunchKernelEx(&cfg, chunk_join_kernel<T, 128>, p, rows)
                       : cudaLaunchKernelEx(&cfg, chunk_join_kernel<T, 64>, p, rows);
}

}  // namespace

cudaError_t launch_chunk_join(DType dt, int kernel_d, int rows, const ChunkParams& p, int num_sms,
                              cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_typed<float>(kernel_d, rows, p, num_sms, stream);
    case kF16: return launch_typed<__half>(kernel_d, rows, p, num_sms, stream);
    case kBF16: return launch_typed<__nv_bfloat16>(kernel_d, rows, p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jvp
