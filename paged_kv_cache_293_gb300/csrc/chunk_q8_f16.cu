// chunk_q8_f16.cu -- instantiates the chunk attention kernel for __half queries over 8-bit pools.
#include "chunk.cuh"

namespace pkv {

template <>
cudaError_t launch_chunk_q8<__half>(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                                cudaStream_t stream) {
    return launch_chunk_impl<__half, true>(plan, p, x, stream);
}

}  // namespace pkv
