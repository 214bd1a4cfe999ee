// chunk_join.cu -- joins the pieces of cut items of the attention of chunks: per
// row, partial outputs weighted by their log-sum-exps, in the order of the keys.
//
// The first part of a cut item lies in the second slot of the CTA that began it, the
// others in the first slots of the CTAs behind.  A warp takes four rows at a
// time, whose parts it loads together; a block takes 32 rows of a CTA's cut item.
#include <cmath>

#include "debug_checks.cuh"
#include "rows.cuh"
#include "serve_internal.h"

namespace jvp {
namespace {

constexpr int kJoinWarps = 8, kJoinRows = 4;  // rows of a warp at once
constexpr int kUnit = kJoinWarps * kJoinRows;  // rows of a block

template <typename T, int DPAD>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const ChunkParams p, int rows) {
  constexpr int C = DPAD / 32, R = kJoinRows;  // columns of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_rows = rows / p.query_tiles, per = rows / kUnit;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x / per;
  const int4 item = p.ws_item[cta];  // CTAs, first row, tokens, head
  if (item.x == 0) return;
  const int hk = item.w / p.head_blocks;
  const int head0 = (item.w - hk * p.head_blocks) * p.group_rows;
  const int row0 = blockIdx.x % per * kUnit + warp * R;
  int token[R], in_group[R];
  bool on[R], any = false;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int x = (row0 + k) / tile_rows, r = row0 + k - x * tile_rows;
    const int rt = r / p.group_rows;
    token[k] = x * p.tok + rt, in_group[k] = head0 + r - rt * p.group_rows;
    on[k] = rt < p.tok && token[k] < item.z && in_group[k] < p.group;
    any |= on[k];
  }
  if (!any) return;  // uniform over the warp
  float M[R], L[R], acc[R][C];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    M[k] = -INFINITY, L[k] = 0.f;
#pragma unroll
    for (int d = 0; d < C; ++d) acc[k][d] = 0.f;
  }
#pragma unroll 2
  for (int i = 0; i < item.x; ++i) {
    const long long at = (2ll * (cta + i) + (i == 0 ? 1 : 0)) * rows + row0;
    float y[R], v[R][C];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      y[k] = -INFINITY;
#pragma unroll
      for (int d = 0; d < C; ++d) v[k][d] = 0.f;
      if (!on[k] || !JVP_CHECK(at + k < 2ll * p.grid * rows, p.c.status, kChkGlobalRow)) continue;
      y[k] = p.ws_lse[at + k];
      if constexpr (C == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p.ws_o + (at + k) * DPAD + lane * C);
        v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
      } else {
        const float2 w = *reinterpret_cast<const float2*>(p.ws_o + (at + k) * DPAD + lane * C);
        v[k][0] = w.x, v[k][1] = w.y;
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float m = fmaxf(M[k], y[k]), mu = m == -INFINITY ? 0.f : m;
      const float a = exp2f(M[k] - mu), w = exp2f(y[k] - mu);
      M[k] = m;
      L[k] = L[k] * a + w;
#pragma unroll
      for (int d = 0; d < C; ++d) acc[k][d] = fmaf(w, v[k][d], acc[k][d] * a);
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (!on[k]) continue;
    const float inv = L[k] == 0.f ? 0.f : 1.f / L[k];
    const int h = hk * p.group + in_group[k];
    const long long t = static_cast<long long>(item.y) + token[k];
    if (!JVP_CHECK(t < p.T && h < p.H, p.c.status, kChkGlobalRow)) continue;
    T* dst = static_cast<T*>(p.o) + t * p.so.n + h * p.so.h;
#pragma unroll
    for (int d = 0; d < C; ++d)
      if (lane * C + d < p.c.D) dst[lane * C + d] = Rows<T>::put(acc[k][d] * inv);
    if (lane == 0 && p.lse)
      p.lse[h * static_cast<long long>(p.T) + t] =
          L[k] == 0.f ? -INFINITY : (M[k] + log2f(L[k])) * 0.6931471805599453f;
  }
}

template <typename T>
cudaError_t launch_typed(int kernel_d, int rows, const ChunkParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.grid * (rows / kUnit));
  return kernel_d > 64
             ? launch_dependent(chunk_join_kernel<T, 128>, grid, kJoinWarps * 32, 0, stream, p, rows)
             : launch_dependent(chunk_join_kernel<T, 64>, grid, kJoinWarps * 32, 0, stream, p, rows);
}

}  // namespace

cudaError_t launch_chunk_join(DType dt, int kernel_d, int rows, const ChunkParams& p,
                              cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_typed<float>(kernel_d, rows, p, stream);
    case kF16: return launch_typed<__half>(kernel_d, rows, p, stream);
    case kBF16: return launch_typed<__nv_bfloat16>(kernel_d, rows, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jvp
