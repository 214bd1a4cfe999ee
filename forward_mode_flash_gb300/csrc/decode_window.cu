// decode_window.cu -- single tokens over the keys of a window and the sinks.
#include "decode.cuh"

namespace jvp {

cudaError_t launch_decode_window(DType dt, bool e4m3, bool tc, bool vec, const DecodeParams& p,
                                 cudaStream_t stream) {
  return launch_any<true>(dt, e4m3, tc, vec, p, stream);
}

}  // namespace jvp
