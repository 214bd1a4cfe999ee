// rows.cuh -- conversions of the element types of packed and cached rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace jvp {

template <typename T>
struct Rows;  // conversions of a row's element type
template <>
struct Rows<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Rows<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Rows<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

}  // namespace jvp
