// chunk_simt.cu -- attention of chunks over a paged cache on the CUDA cores: fp32
// arithmetic, any element type, any head dimension up to 128, any alignment and
// page size.
//
// The products and the softmax are those of the kernel over packed prompts
// (packed_simt.cu): 32 query rows against 64-key tiles in shared memory, a thread
// forming 4 x 4 pieces of S and 4 x D/16 pieces of O by paired FMAs.  A tile's rows
// are tokens times the query heads of a key/value head, so a few tokens still fill
// it; its keys' places are looked up by one thread each, a tile ahead; the work is
// divided among the blocks as on the tensor cores (chunk.cuh).  Bound by the reads of
// shared memory on long chunks (fp32, 2 chunks of 2000 tokens over 4096 positions, 8/2
// heads of 64: 796 us, 32 TFLOP/s), by a tile's latency, 3 us, on short ones.
#include <cmath>
#include <type_traits>

#include "chunk.cuh"
#include "rows.cuh"
#include "sm103_ptx.cuh"

namespace jvp {
namespace {

constexpr int kThreads = 128, TY = kThreads / 16;
constexpr int BM = kChunkSimtRows, BN = kChunkSimtTile;
static_assert(BM == 4 * TY, "four rows per thread");

template <int DP>
struct Smem {
  static constexpr int LD = DP + 4;  // Q and K rows
  static constexpr int LP = BN + 4;  // P rows
  static constexpr int Q = 0, K = Q + BM * LD, V = K + BN * LD, P = V + BN * DP;
  static constexpr int FLOATS = P + BM * LP;
};
// Places of a tile's keys (elements from the start of the cache, -1: no such key)
// and their scales.
struct Places {
  long long k[BN], v[BN];
  float ks[BN], vs[BN];
};

// Four columns from d of a row, zeros past D.
template <typename TC>
__device__ __forceinline__ float element(const TC* x) {
  return Rows<TC>::get(*x);
}
template <>
__device__ __forceinline__ float element<uint8_t>(const uint8_t* x) {
  const uint32_t h2 = e4m3x2_to_half2(*x);
  return __half22float2(*reinterpret_cast<const __half2*>(&h2)).x;
}
template <typename TC>
__device__ __forceinline__ float4 four(const TC* row, int d, int D, bool vec) {
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) {  // (D is a multiple of 4)
    if (d >= D) return f;
    if constexpr (sizeof(TC) == 4) {
      f = __ldg(reinterpret_cast<const float4*>(row + d));
    } else if constexpr (sizeof(TC) == 2) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + d));
      const TC* e = reinterpret_cast<const TC*>(&w);
      f = make_float4(element(e), element(e + 1), element(e + 2), element(e + 3));
    } else {
      uint32_t a, b;
      e4m3x4_to_half2x2(__ldg(reinterpret_cast<const uint32_t*>(row + d)), a, b);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
      f = make_float4(x.x, x.y, y.x, y.y);
    }
    return f;
  }
  if (d < D) f.x = element(row + d);
  if (d + 1 < D) f.y = element(row + d + 1);
  if (d + 2 < D) f.z = element(row + d + 2);
  if (d + 3 < D) f.w = element(row + d + 3);
  return f;
}

template <typename T, int DP, bool E4M3>
__global__ void __launch_bounds__(kThreads) chunk_simt_kernel(const __grid_constant__ ChunkParams p) {
  using L = Smem<DP>;
  using TC = typename std::conditional<E4M3, uint8_t, T>::type;
  constexpr bool kCopy = sizeof(TC) == 4;  // 16-byte pieces go to shared memory as they are
  constexpr int DC = DP / 16;              // output columns per thread: 4 tx + 64 e .. + 3
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm + L::Q, *sK = sm + L::K, *sV = sm + L::V, *sP = sm + L::P;
  __shared__ Places places[2];
  const PagedCache& c = p.c;
  const bool vec = p.vec != 0;
  const int tid = static_cast<int>(threadIdx.x), tx = tid & 15, ty = tid >> 4;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ChunkSpan span;
  static_assert(sizeof(ChunkScratch) <= L::FLOATS * 4, "the tiles' space");
  if (!chunk_divide<BN, kThreads>(p, reinterpret_cast<ChunkScratch*>(sm), &span)) return;
  if (p.cut && tid == 0) chunk_name<BN>(p, span);
  ChunkWalk<BN> walk(p, span.start, span.end);
  ChunkPart<BN> it;
  while (walk.next(p, &it)) {
    const int hk = it.head / p.head_blocks, hb = it.head - hk * p.head_blocks;
    const int toks = it.toks, t0 = it.t0, t1 = it.t1, slot = it.slot;
    const ChunkKeys<BN>& keys = it.see;

    // token (of the item) and query head of row r; -1: no such row
    auto token_of = [&](int r) {
      const int t = r / p.group_rows, h = hb * p.group_rows + r - t * p.group_rows;
      return t < toks && h < p.group ? t : -1;
    };
    auto head_of = [&](int r) { return hk * p.group + hb * p.group_rows + r % p.group_rows; };
    auto look_up = [&](int t) {
      if (t >= t1 || tid >= BN) return;
      Places& to = places[t & 1];
      const int j = keys.tile(t) * BN + tid;
      to.k[tid] = to.v[tid] = -1;
      if (keys.unseen(j, 1) || j >= it.keys) return;
      int entry, row;
      split_position(c, j, &entry, &row);
      const int page = page_of(c, it.b, entry);
      if (page < 0) return;
      to.k[tid] = page * c.sk.b + hk * c.sk.h + row * c.sk.n;
      to.v[tid] = page * c.sv.b + hk * c.sv.h + row * c.sv.n;
      if constexpr (E4M3) {
        const long long at = (static_cast<long long>(page) * c.Hkv + hk) * c.page_size + row;
        to.ks[tid] = scale_value(__ldg(c.k_scale + at));
        to.vs[tid] = scale_value(__ldg(c.v_scale + at));
      }
    };
    // a tile's rows into shared memory; zeros for keys that are not there
    auto load_rows = [&](float* dst, int ld, const TC* base, const long long* at, const float* scale) {
      for (int e = tid; e < BN * (DP / 4); e += kThreads) {
        const int row = e / (DP / 4), d = 4 * (e % (DP / 4));
        const long long place = at[row];
        float* to = dst + row * ld + d;
        if (kCopy && vec) {
          const bool on = place >= 0 && d < c.D;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                       "l"(base + (on ? place + d : 0)), "r"(on ? 16 : 0)
                       : "memory");
        } else {
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
          if (place >= 0) {
            f = four(base + place, d, c.D, vec);
            if constexpr (E4M3) f.x *= scale[row], f.y *= scale[row], f.z *= scale[row], f.w *= scale[row];
          }
          *reinterpret_cast<float4*>(to) = f;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load_k = [&](int t) {
      load_rows(sK, L::LD, static_cast<const TC*>(c.k), places[t & 1].k, places[t & 1].ks);
    };
    auto load_v = [&](int t) {
      load_rows(sV, DP, static_cast<const TC*>(c.v), places[t & 1].v, places[t & 1].vs);
    };
    __syncthreads();  // the last part's tiles have been read
    look_up(t0);
    for (int e = tid; e < BM * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), d = 4 * (e % (DP / 4)), t = token_of(r);
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t >= 0)
        f = four(static_cast<const T*>(p.q) + static_cast<long long>(it.r0 + it.tok0 + t) * p.sq.n +
                     static_cast<long long>(head_of(r)) * p.sq.h,
                 d, c.D, false);
      *reinterpret_cast<float4*>(sQ + r * L::LD + d) = f;
    }
    __syncthreads();
    load_k(t0);
    load_v(t0);
    int at[4], lo[4];  // positions of the thread's rows (-1: no such row), their windows
    float m[4], l[4], acc[4][DC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = token_of(ty + TY * i);
      at[i] = t < 0 ? -1 : it.past + it.tok0 + t;
      lo[i] = keys.lo(at[i]);
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < DC; ++e) acc[i][e] = 0.f;
    }
    auto sees = [&](int i, int j) { return j <= at[i] && (j >= lo[i] || j < keys.sinks); };
    for (int t = t0; t < t1; ++t) {
      const int j0 = keys.tile(t) * BN;
      look_up(t + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // K; V may be on its way
      __syncthreads();
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
      for (int i = 0; i < 4; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = tx + 16 * j;
          s[i][j] = sees(i, j0 + col) && places[t & 1].k[col] >= 0
                        ? (s2[i][j].x + s2[i][j].y) * p.scale_log2
                        : -INFINITY;
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
      asm volatile("cp.async.wait_group 0;" ::: "memory");  // V
      __syncthreads();  // P is written, V has landed, K has been read
      if (t + 1 < t1) load_k(t + 1);
      // acc += P V.  In a tile that a mask cuts, a masked key's weight is 0 and its
      // values are left out (0 * NaN would not be 0).
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
                if (masked.value && !sees(i, j0 + j + jj)) continue;
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
      if (j0 + BN - 1 > it.past + it.tok0 || j0 < keys.lo_last) values(std::true_type());
      else values(std::false_type());
      __syncthreads();  // V and P have been read
      if (t + 1 < t1) load_v(t + 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      const int r = ty + TY * i, t = token_of(r);
      if (t < 0) continue;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      const float lse2 = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
      const long long row = static_cast<long long>(it.r0) + it.tok0 + t;
      const int h = head_of(r);
      const long long ws = static_cast<long long>(slot) * BM + r;
      if (slot >= 0 && !JVP_CHECK(slot < 2 * p.grid, c.status, kChkGlobalRow)) continue;
      if (tx == 0) {
        if (slot >= 0) p.ws_lse[ws] = lse2;
        else if (p.lse) p.lse[static_cast<long long>(h) * p.T + row] = lse2 * 0.6931471805599453f;
      }
      T* dst = static_cast<T*>(p.o) + row * p.so.n + h * p.so.h;
#pragma unroll
      for (int e = 0; e < DC; ++e) {
        const int d = 4 * tx + 16 * (e & ~3) + (e & 3);
        if (slot >= 0) p.ws_o[ws * DP + d] = acc[i][e] * inv;
        else if (d < c.D) dst[d] = Rows<T>::put(acc[i][e] * inv);
      }
    }
  }
}

template <typename T, int DP, bool E4M3>
cudaError_t launch_variant(const ChunkParams& p, cudaStream_t stream) {
  constexpr int bytes = Smem<DP>::FLOATS * 4;
  const cudaError_t e = allow_shared_memory<chunk_simt_kernel<T, DP, E4M3>>(bytes);
  if (e != cudaSuccess) return e;
  chunk_simt_kernel<T, DP, E4M3>
      <<<static_cast<unsigned>(p.grid), kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_typed(bool e4m3, const ChunkParams& p, cudaStream_t stream) {
  if (p.c.D > 64)
    return e4m3 ? launch_variant<T, 128, true>(p, stream) : launch_variant<T, 128, false>(p, stream);
  return e4m3 ? launch_variant<T, 64, true>(p, stream) : launch_variant<T, 64, false>(p, stream);
}

}  // namespace

cudaError_t launch_chunk_simt(DType dt, bool e4m3, const ChunkParams& p, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_typed<float>(e4m3, p, stream);
    case kF16: return launch_typed<__half>(e4m3, p, stream);
    case kBF16: return launch_typed<__nv_bfloat16>(e4m3, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jvp
