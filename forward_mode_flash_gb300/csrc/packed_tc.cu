// packed_tc.cu -- instantiations of the tensor-core kernel over packed prompts.
#include "packed_tc.cuh"

namespace jvp {

template <typename T>
static cudaError_t launch_typed(int kernel_d, const PackedMaps& maps, const PackedParams& p,
                                cudaStream_t stream) {
  if (kernel_d == 64)
    return p.query_tiles == 1 ? launch_packed_tc_variant<T, 64, 1>(maps, p, stream)
                              : launch_packed_tc_variant<T, 64, 2>(maps, p, stream);
  return p.query_tiles == 1 ? launch_packed_tc_variant<T, 128, 1>(maps, p, stream)
                            : launch_packed_tc_variant<T, 128, 2>(maps, p, stream);
}

cudaError_t launch_packed_tc(DType dt, int kernel_d, const PackedMaps& maps, const PackedParams& p,
                             cudaStream_t stream) {
  return dt == kF16 ? launch_typed<__half>(kernel_d, maps, p, stream)
                    : launch_typed<__nv_bfloat16>(kernel_d, maps, p, stream);
}

}  // namespace jvp
