// decode.cu -- single tokens over all their cached keys.
#include "decode.cuh"

namespace jvp {

cudaError_t launch_decode(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
                          cudaStream_t stream) {
  return launch_any<false>(dt, e4m3, tc, vec, p, stream);
}

}  // namespace jvp
