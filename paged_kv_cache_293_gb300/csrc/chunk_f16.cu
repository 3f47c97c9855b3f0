// chunk_f16.cu -- instantiates the chunk attention kernel for __half pools.
#include "chunk.cuh"

namespace pkv {

template <>
cudaError_t launch_chunk<__half>(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                                 cudaStream_t stream) {
    return launch_chunk_impl<__half>(plan, p, x, stream);
}

}  // namespace pkv
