// chunk_tc.cu -- instantiations of the tensor-core kernel over a paged cache.
#include "chunk_tc.cuh"

namespace jvp {

template <typename T, ChunkSource SRC>
static cudaError_t launch_typed(int kernel_d, const ChunkMaps& maps, const ChunkParams& p,
                                cudaStream_t stream) {
  // (the gathering warps leave registers and shared memory for one CTA per SM)
  if constexpr (SRC == kChunkBoxes) {
    if (p.query_tiles == 1)
      return kernel_d == 64 ? launch_chunk_tc_variant<T, 64, 1, SRC>(maps, p, stream)
                            : launch_chunk_tc_variant<T, 128, 1, SRC>(maps, p, stream);
  }
  return kernel_d == 64 ? launch_chunk_tc_variant<T, 64, 2, SRC>(maps, p, stream)
                        : launch_chunk_tc_variant<T, 128, 2, SRC>(maps, p, stream);
}

template <typename T>
static cudaError_t launch_source(int kernel_d, ChunkSource source, const ChunkMaps& maps,
                                 const ChunkParams& p, cudaStream_t stream) {
  switch (source) {
    case kChunkBoxes: return launch_typed<T, kChunkBoxes>(kernel_d, maps, p, stream);
    case kChunkRows: return launch_typed<T, kChunkRows>(kernel_d, maps, p, stream);
    case kChunkE4M3: return launch_typed<T, kChunkE4M3>(kernel_d, maps, p, stream);
    case kChunkStaged: return launch_typed<T, kChunkStaged>(kernel_d, maps, p, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_chunk_tc(DType dt, int kernel_d, ChunkSource source, const ChunkMaps& maps,
                            const ChunkParams& p, cudaStream_t stream) {
  return dt == kF16 ? launch_source<__half>(kernel_d, source, maps, p, stream)
                    : launch_source<__nv_bfloat16>(kernel_d, source, maps, p, stream);
}

}  // namespace jvp
