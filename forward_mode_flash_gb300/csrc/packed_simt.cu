// packed_simt.cu -- attention over packed prompts on the CUDA cores: fp32
// arithmetic, any element type, any head dimension up to 128, any alignment.
//
// The same online softmax as the tensor-core kernel.  A block of 128 threads
// takes 32 query rows of one head against 64-key tiles in shared memory; a
// thread forms a 4 x 4 piece of S (rows ty + 8 i, keys tx + 16 j: 16-byte reads
// along the head dimension, K rows padded by 4 floats so that 16 lanes' rows
// hit distinct banks) and then a 4 x D/16 piece of O.  Either product reads
// 8 x 16 bytes of shared memory for 64 FMAs.  Bound by fp32 FMA issue.
// float32 tiles are copied asynchronously, K's next tile during the softmax
// and the second product, V's during the next scores; four blocks per SM (two
// at D > 64) overlap the rest.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "packed.cuh"

namespace jvp {
namespace {

constexpr int kThreads = 128;
constexpr int BM = kPackedSimtRows, BN = 64, TY = kThreads / 16;
static_assert(BM == 4 * TY, "four rows per thread");

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

template <int DP>
struct Smem {
  static constexpr int LD = DP + 4;  // Q and K rows
  static constexpr int LP = BN + 4;  // P rows
  static constexpr int Q = 0, K = Q + BM * LD, V = K + BN * LD, P = V + BN * DP;
  static constexpr int FLOATS = P + BM * LP;
};

// VEC: float rows that are 16-byte aligned, D a multiple of 4.
template <typename T, int DP, bool VEC>
__global__ void __launch_bounds__(kThreads) packed_simt_kernel(const PackedParams p) {
  using L = Smem<DP>;
  constexpr int DC = DP / 16;  // output columns per thread: 4 tx + 64 e .. + 3
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm + L::Q, *sK = sm + L::K, *sV = sm + L::V, *sP = sm + L::P;
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

  // rows [row0, row0 + ROWS) of a tensor into shared memory (leading dimension
  // ld): zeros past D and for rows that do not exist
  auto load_rows = [&](float* dst, int ld, int rows, const T* base, long long stride, int row0) {
    for (int e = tid; e < rows * (DP / 4); e += kThreads) {
      const int row = e / (DP / 4), d = 4 * (e % (DP / 4));
      const bool on = row0 + row < len && d < p.D;
      const T* src = base + (on ? (row0 + row) * stride + d : 0);
      float* to = dst + row * ld + d;
      if constexpr (VEC) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                     "l"(src), "r"(on ? 16 : 0)
                     : "memory");
      } else {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (on && d + i < p.D) ? to_f(src[i]) : 0.f;
        *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
    if (VEC) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // all but the latest group of copies have landed / all have
  auto wait_but_latest = [&]() {
    if (VEC) asm volatile("cp.async.wait_group 1;" ::: "memory");
  };
  auto wait_all = [&]() {
    if (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
  };
  load_rows(sQ, L::LD, BM, q, p.sq.n, q0);
  load_rows(sK, L::LD, BN, k, p.sk.n, 0);
  load_rows(sV, DP, BN, v, p.sv.n, 0);
  float m[4], l[4], acc[4][DC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DC; ++e) acc[i][e] = 0.f;
  }
  for (int j0 = 0; j0 < keys; j0 += BN) {
    wait_but_latest();  // K (and Q); V may be on its way
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = *reinterpret_cast<const float4*>(sQ + (ty + TY * i) * L::LD + d);
        b[i] = *reinterpret_cast<const float4*>(sK + (tx + 16 * i) * L::LD + d);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
          s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
          s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
          s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = q0 + ty + TY * i;
      const int limit = p.causal ? min(row + 1, len) : len;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (j0 + tx + 16 * j < limit) ? s[i][j] * p.scale_log2 : -INFINITY;
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
        sP[(ty + TY * i) * L::LP + tx + 16 * j] = s[i][j];
      }
      l[i] = l[i] * a + sum;  // this thread's keys
#pragma unroll
      for (int e = 0; e < DC; ++e) acc[i][e] *= a;
    }
    wait_all();       // V
    __syncthreads();  // P is written, V has landed, K has been read
    const bool more = j0 + BN < keys;
    if (more) load_rows(sK, L::LD, BN, k, p.sk.n, j0 + BN);
    // acc += P V.  In a tile that the causal mask cuts, a masked key's weight
    // is 0 and its values are left out (0 * NaN would not be 0).
    auto values = [&](auto masked) {
#pragma unroll 2
      for (int j = 0; j < BN; j += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = *reinterpret_cast<const float4*>(sP + (ty + TY * i) * L::LP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
          for (int e = 0; e < DC; e += 4) {
            const float4 b = *reinterpret_cast<const float4*>(sV + (j + jj) * DP + 4 * tx + 16 * e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (masked.value && j0 + j + jj > q0 + ty + TY * i) continue;
              const float w = jj == 0 ? a[i].x : jj == 1 ? a[i].y : jj == 2 ? a[i].z : a[i].w;
              acc[i][e] = fmaf(w, b.x, acc[i][e]);
              acc[i][e + 1] = fmaf(w, b.y, acc[i][e + 1]);
              acc[i][e + 2] = fmaf(w, b.z, acc[i][e + 2]);
              acc[i][e + 3] = fmaf(w, b.w, acc[i][e + 3]);
            }
          }
      }
    };
    if (p.causal && j0 + BN - 1 > q0) values(std::true_type());
    else values(std::false_type());
    __syncthreads();  // V and P have been read
    if (more) load_rows(sV, DP, BN, v, p.sv.n, j0 + BN);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + TY * i;
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
  constexpr int bytes = Smem<DP>::FLOATS * 4;
  const cudaError_t e = allow_shared_memory<packed_simt_kernel<T, DP, VEC>>(bytes);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.tiles) * p.H;
  packed_simt_kernel<T, DP, VEC><<<static_cast<unsigned>(grid), kThreads, bytes, stream>>>(p);
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
