// chunk_tc.cu -- instantiations of the tensor-core kernel over a paged cache.
#include "chunk_tc.cuh"

namespace jvp {

template <typename T, ChunkSource SRC>
static cudaError_t launch_typed(int kernel_d, const ChunkMaps& maps, const ChunkParams& p,
                                cudaStream_t stream) {
  if (kernel_d == 64)
    return p.query_tiles == 1 ? launch_chunk_tc_variant<T, 64, 1, SRC>(maps, p, stream)
                              : launch_chunk_tc_variant<T, 64, 2, SRC>(maps, p, stream);
  return p.query_tiles == 1 ? launch_chunk_tc_variant<T, 128, 1, SRC>(maps, p, stream)
                            : launch_chunk_tc_variant<T, 128, 2, SRC>(maps, p, stream);
}

cudaError_t launch_chunk_tc(DType dt, int kernel_d, ChunkSource source, const ChunkMaps& maps,
                            const ChunkParams& p, cudaStream_t stream) {
  if (source != kChunkBoxes) return cudaErrorInvalidValue;
  return dt == kF16 ? launch_typed<__half, kChunkBoxes>(kernel_d, maps, p, stream)
                    : launch_typed<__nv_bfloat16, kChunkBoxes>(kernel_d, maps, p, stream);
}

}  // namespace jvp
