// packed_simt.cu -- attention over packed prompts on the CUDA cores: fp32
// arithmetic, any element type, any head dimension up to 128, any alignment.
//
// The same online softmax as the tensor-core kernel.  A block takes 32 query rows
// of one head against 64-key tiles in shared memory, with 128 threads or with
// two halves of 128 that take every other key tile and join at the end (so that
// the block with most keys ends sooner).  A thread forms a 4 x 4 piece of S
// (rows ty + 8 i, keys tx + 16 j: 16-byte reads along the head dimension, K rows
// padded by 4 floats so that 16 lanes' rows hit distinct banks) and then a
// 4 x D/16 piece of O.  Either product reads 8 x 16 bytes of shared memory for
// 64 FMAs, issued as pairs (10 % less time: the rest of the loop wants the issue
// slots).  Bound by those reads (on long prompts the shared-memory pipe is 69 %
// active, the FMA pipe 55 %).  float32 tiles are copied asynchronously,
// K's next tile during the softmax and the second product, V's during the next
// scores.  Measured, causal: eight prompts of about 1000 tokens, 8/8 heads of
// 64: 273 us, 31 TFLOP/s of counted products (those of tiles that the mask cuts
// are formed whole); four of 125 to 700 tokens, 8/2 heads of 64: 55 us, where
// the FMAs alone take 13 (the last wave is short).  16-bit rows that the tensor
// cores cannot take (converted while they are loaded, not copied): bf16, eight of
// 1024 tokens, 8/8 heads of 60: 355 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "packed.cuh"
#include "sm103_ptx.cuh"

namespace jvp {
namespace {

constexpr int kHalf = 128;  // threads of a half
constexpr int BM = kPackedSimtRows, BN = 64, TY = kHalf / 16;
static_assert(BM == 4 * TY, "four rows per thread");

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

template <int DP, int HALVES>
struct Smem {
  static constexpr int LD = DP + 4;  // Q and K rows
  static constexpr int LP = BN + 4;  // P rows
  // (of a half, behind Q) and what a half leaves for the other
  static constexpr int Q = 0, K = 0, V = K + BN * LD, P = V + BN * DP, HALF = P + BM * LP;
  static constexpr int FLOATS = BM * LD + HALVES * HALF;
  static_assert(BM * (DP + 2) <= HALF, "a half's state fits");
};

// VEC: float rows that are 16-byte aligned, D a multiple of 4.
template <typename T, int DP, bool VEC, int HALVES>
__global__ void __launch_bounds__(HALVES* kHalf) packed_simt_kernel(const PackedParams p) {
  using L = Smem<DP, HALVES>;
  constexpr int DC = DP / 16;  // output columns per thread: 4 tx + 64 e .. + 3
  extern __shared__ __align__(16) float sm[];
  const int half = HALVES == 1 ? 0 : static_cast<int>(threadIdx.x) / kHalf;
  float* const mine = sm + BM * L::LD + half * L::HALF;
  float *sQ = sm + L::Q, *sK = mine + L::K, *sV = mine + L::V, *sP = mine + L::P;
  const int h = static_cast<int>(blockIdx.x) / p.tiles, hk = h / p.group;
  const int u = static_cast<int>(blockIdx.x) % p.tiles;
  PackedTile pt;
  if (!find_packed_tile(p.cu, p.B, p.T, BM, u, p.causal != 0, p.status, &pt)) return;
  const int len = pt.len, q0 = pt.tile * BM;
  const int keys = p.causal ? min(q0 + BM, len) : len;
  const int tid = static_cast<int>(threadIdx.x) % kHalf, tx = tid & 15, ty = tid >> 4;
  auto sync_half = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(kHalf) : "memory"); };
  const T* q = static_cast<const T*>(p.q) + pt.r0 * p.sq.n + h * p.sq.h;
  const T* k = static_cast<const T*>(p.k) + pt.r0 * p.sk.n + hk * p.sk.h;
  const T* v = static_cast<const T*>(p.v) + pt.r0 * p.sv.n + hk * p.sv.h;

  // rows [row0, row0 + ROWS) of a tensor into shared memory (leading dimension
  // ld): zeros past D and for rows that do not exist
  auto load_rows = [&](float* dst, int ld, int rows, const T* base, long long stride, int row0) {
    for (int e = tid; e < rows * (DP / 4); e += kHalf) {
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
  constexpr int QR = BM / HALVES;
  load_rows(sQ + half * QR * L::LD, L::LD, QR, q, p.sq.n, q0 + half * QR);
  if (half * BN < keys) {
    load_rows(sK, L::LD, BN, k, p.sk.n, half * BN);
    load_rows(sV, DP, BN, v, p.sv.n, half * BN);
    wait_but_latest();
  } else {
    wait_all();
  }
  __syncthreads();  // Q
  float m[4], l[4], acc[4][DC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DC; ++e) acc[i][e] = 0.f;
  }
  for (int j0 = half * BN; j0 < keys; j0 += HALVES * BN) {
    wait_but_latest();  // K; V may be on its way
    sync_half();
    float s[4][4];
    float2 s2[4][4];  // sums over the even and the odd columns
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
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
          s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s2[i][j]);
          s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s2[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
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
    wait_all();   // V
    sync_half();  // P is written, V has landed, K has been read
    const int next = j0 + HALVES * BN;
    if (next < keys) load_rows(sK, L::LD, BN, k, p.sk.n, next);
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
              const float2 ww = make_float2(w, w);
              const float2 y0 = fma2(ww, make_float2(b.x, b.y), make_float2(acc[i][e], acc[i][e + 1]));
              const float2 y1 =
                  fma2(ww, make_float2(b.z, b.w), make_float2(acc[i][e + 2], acc[i][e + 3]));
              acc[i][e] = y0.x, acc[i][e + 1] = y0.y, acc[i][e + 2] = y1.x, acc[i][e + 3] = y1.y;
            }
          }
      }
    };
    if (p.causal && j0 + BN - 1 > q0) values(std::true_type());
    else values(std::false_type());
    sync_half();  // V and P have been read
    if (next < keys) load_rows(sV, DP, BN, v, p.sv.n, next);
  }
  // The other half's state joins this one's: a thread's own numbers, thread by
  // thread.
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  if constexpr (HALVES == 2) {
    float* const left = mine + (1 - half) * L::HALF + tid;  // half 1's space
    float* const stats = mine + (1 - half) * L::HALF + BM * DP;
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < DC; ++e) left[(i * DC + e) * kHalf] = acc[i][e];
        if (tx == 0) stats[ty + TY * i] = m[i], stats[BM + ty + TY * i] = l[i];
      }
    }
    __syncthreads();
    if (half == 1) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mo = stats[ty + TY * i], M = fmaxf(m[i], mo), mu = M == -INFINITY ? 0.f : M;
      const float a = exp2f(m[i] - mu), b = exp2f(mo - mu);
      l[i] = l[i] * a + stats[BM + ty + TY * i] * b;
      m[i] = M;
#pragma unroll
      for (int e = 0; e < DC; ++e) acc[i][e] = acc[i][e] * a + left[(i * DC + e) * kHalf] * b;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + TY * i;
    if (row >= len) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    if (tx == 0 && p.lse)
      p.lse[static_cast<long long>(h) * p.T + pt.r0 + row] =
          l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
    T* dst = static_cast<T*>(p.o) + static_cast<long long>(pt.r0 + row) * p.so.n + h * p.so.h;
#pragma unroll
    for (int e = 0; e < DC; ++e) {
      const int d = 4 * tx + 16 * (e & ~3) + (e & 3);
      if (d < p.D) from_f(dst[d], acc[i][e] * inv);
    }
  }
}

template <typename T, int DP, bool VEC, int HALVES>
cudaError_t launch_variant(const PackedParams& p, cudaStream_t stream) {
  constexpr int bytes = Smem<DP, HALVES>::FLOATS * 4;
  const cudaError_t e = allow_shared_memory<packed_simt_kernel<T, DP, VEC, HALVES>>(bytes);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.tiles) * p.H;
  packed_simt_kernel<T, DP, VEC, HALVES>
      <<<static_cast<unsigned>(grid), HALVES * kHalf, bytes, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, bool VEC>
cudaError_t launch_typed(const PackedParams& p, cudaStream_t stream) {
  // Two halves where an average prompt has more than one key tile and two
  // blocks fit on an SM (fp32, 8/2 heads of 64, four of 125 to 700 tokens: 55
  // us with two halves, 66 with one; 16 prompts of up to 60 tokens, D = 128: 17
  // and 12.5; 16/4 heads of 128, four of about 1000 tokens: 623 and 598).
  if (p.D > 64) return launch_variant<T, 128, VEC, 1>(p, stream);
  return p.T > static_cast<long long>(BN) * p.B ? launch_variant<T, 64, VEC, 2>(p, stream)
                                                : launch_variant<T, 64, VEC, 1>(p, stream);
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
