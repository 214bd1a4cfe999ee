// packed_tc.cu -- instantiations of the tensor-core kernel over packed prompts.
#include "packed_tc.cuh"

namespace jvp {

cudaError_t launch_packed_tc(DType dt, int kernel_d, const PackedMaps& maps, const PackedParams& p,
                             cudaStream_t stream) {
  if (dt == kF16)
    return kernel_d == 64 ? launch_packed_tc_variant<__half, 64>(maps, p, stream)
                          : launch_packed_tc_variant<__half, 128>(maps, p, stream);
  return kernel_d == 64 ? launch_packed_tc_variant<__nv_bfloat16, 64>(maps, p, stream)
                        : launch_packed_tc_variant<__nv_bfloat16, 128>(maps, p, stream);
}

}  // namespace jvp
