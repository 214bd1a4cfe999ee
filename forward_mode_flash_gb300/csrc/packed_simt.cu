// packed_simt.cu -- attention over packed prompts on the CUDA cores: fp32
// arithmetic, any element type, any head dimension up to 128, any alignment.
//
// The same online softmax as the tensor-core kernel.  A block of 256 threads
// takes 64 query rows of one head against 64-key tiles: Q and K are held
// transposed in shared memory ([d][row]), so a thread forms a 4 x 4 piece of
// S from two 16-byte reads per column of the head dimension, and after the
// softmax a 4 x D/16 piece of O from the transposed P.  Bound by fp32 FMA
// issue: 16 FMAs against two shared-memory reads in the first product, 4 D/16
// against 1 + D/64 in the second.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "packed.cuh"

namespace jvp {
namespace {

constexpr int kThreads = 256;
constexpr int BM = kPackedSimtRows, BN = 64;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

template <int DP>
constexpr int smem_floats() {
  return DP * BM + DP * BN + BN * DP + BN * BM;  // Q^T, K^T, V, P^T
}

// VEC: rows are 16-byte aligned and D is a multiple of 4 (float only).
template <typename T, int DP, bool VEC>
__global__ void __launch_bounds__(kThreads) packed_simt_kernel(const PackedParams p) {
  constexpr int DC = DP / 16;  // output columns per thread: 4 (tx + 16 i) .. + 3
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;             // [DP][BM]
  float* sK = sQ + DP * BM;   // [DP][BN]
  float* sV = sK + DP * BN;   // [BN][DP]
  float* sP = sV + BN * DP;   // [BN][BM]
  const int h = static_cast<int>(blockIdx.x) / p.tiles, hk = h / p.group;
  const int u = static_cast<int>(blockIdx.x) % p.tiles;
  PackedTile pt;
  if (!find_packed_tile(p.cu, p.B, p.T, BM, u, p.causal != 0, p.status, &pt)) return;
  const int len = pt.len, q0 = pt.tile * BM;
  const int keys = p.causal ? min(q0 + BM, len) : len;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const T* q = static_cast<const T*>(p.q) + pt.r0 * p.sq.n + h * p.sq.h;
  const T* k = static_cast<const T*>(p.k) + pt.r0 * p.sk.n + hk * p.sk.h;
  const T* v = static_cast<const T*>(p.v) + pt.r0 * p.sv.n + hk * p.sv.h;

  // four columns from d of a row, zeros past D and for rows that do not exist
  auto load4 = [&](const T* base, long long stride, int row, bool on, int d) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!on || d >= p.D) return f;
    const T* src = base + row * stride + d;
    if constexpr (VEC) {
      f = __ldg(reinterpret_cast<const float4*>(src));
    } else {
      float* e = &f.x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (d + i < p.D) e[i] = to_f(src[i]);
    }
    return f;
  };
  for (int e = tid; e < BM * (DP / 4); e += kThreads) {
    const int row = e % BM, d = 4 * (e / BM);
    const float4 f = load4(q, p.sq.n, q0 + row, q0 + row < len, d);
    sQ[d * BM + row] = f.x, sQ[(d + 1) * BM + row] = f.y;
    sQ[(d + 2) * BM + row] = f.z, sQ[(d + 3) * BM + row] = f.w;
  }
  float m[4], l[4], acc[4][DC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DC; ++e) acc[i][e] = 0.f;
  }
  for (int j0 = 0; j0 < keys; j0 += BN) {
    __syncthreads();  // the previous tile is no longer read
    for (int e = tid; e < BN * (DP / 4); e += kThreads) {
      const int row = e % BN, d = 4 * (e / BN);
      const float4 f = load4(k, p.sk.n, j0 + row, j0 + row < len, d);
      sK[d * BN + row] = f.x, sK[(d + 1) * BN + row] = f.y;
      sK[(d + 2) * BN + row] = f.z, sK[(d + 3) * BN + row] = f.w;
    }
    for (int e = tid; e < BN * (DP / 4); e += kThreads) {
      const int d = 4 * (e % (DP / 4)), row = e / (DP / 4);
      *reinterpret_cast<float4*>(sV + row * DP + d) =
          load4(v, p.sv.n, j0 + row, j0 + row < len, d);
    }
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < DP; ++d) {
      const float4 a = *reinterpret_cast<const float4*>(sQ + d * BM + 4 * ty);
      const float4 b = *reinterpret_cast<const float4*>(sK + d * BN + 4 * tx);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(av[i], bv[j], s[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = q0 + 4 * ty + i;
      const int limit = p.causal ? min(row + 1, len) : len;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (j0 + 4 * tx + j < limit) ? s[i][j] * p.scale_log2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m_new = fmaxf(m[i], top);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float a = exp2f(m[i] - mu);
      m[i] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - mu);
        sum += s[i][j];
      }
      l[i] = l[i] * a + sum;  // this thread's columns
#pragma unroll
      for (int e = 0; e < DC; ++e) acc[i][e] *= a;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(sP + (4 * tx + j) * BM + 4 * ty) =
          make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncthreads();
#pragma unroll 4
    for (int j = 0; j < BN; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(sP + j * BM + 4 * ty);
      const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < DC; e += 4) {
        const float4 b = *reinterpret_cast<const float4*>(sV + j * DP + 4 * tx + 16 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][e] = fmaf(av[i], b.x, acc[i][e]);
          acc[i][e + 1] = fmaf(av[i], b.y, acc[i][e + 1]);
          acc[i][e + 2] = fmaf(av[i], b.z, acc[i][e + 2]);
          acc[i][e + 3] = fmaf(av[i], b.w, acc[i][e + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + 4 * ty + i;
    float sum = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (row >= len) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (tx == 0 && p.lse)
      p.lse[static_cast<long long>(h) * p.T + pt.r0 + row] =
          sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.6931471805599453f;
    T* dst = static_cast<T*>(p.o) + static_cast<long long>(pt.r0 + row) * p.so.n + h * p.so.h;
#pragma unroll
    for (int e = 0; e < DC; ++e) {
      const int d = 4 * tx + 16 * (e & ~3) + (e & 3);
      if (d < p.D) from_f(dst[d], acc[i][e] * inv);
    }
  }
}

template <typename T, int DP, bool VEC>
cudaError_t launch_variant(const PackedParams& p, cudaStream_t stream) {
  constexpr int bytes = smem_floats<DP>() * 4;
  auto kern = packed_simt_kernel<T, DP, VEC>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.tiles) * p.H;
  kern<<<static_cast<unsigned>(grid), kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, bool VEC>
cudaError_t launch_typed(const PackedParams& p, cudaStream_t stream) {
  return p.D <= 64 ? launch_variant<T, 64, VEC>(p, stream) : launch_variant<T, 128, VEC>(p, stream);
}

}  // namespace

cudaError_t launch_packed_simt(DType dt, const PackedParams& p, cudaStream_t stream) {
  switch (dt) {
    case kF32: return p.vec ? launch_typed<float, true>(p, stream) : launch_typed<float, false>(p, stream);
    case kF16: return launch_typed<__half, false>(p, stream);
    case kBF16: return launch_typed<__nv_bfloat16, false>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jvp
