// chunk_bf16.cu -- instantiates the chunk attention kernel for __nv_bfloat16 pools.
#include "chunk.cuh"

namespace pkv {

template <>
cudaError_t launch_chunk<__nv_bfloat16>(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                                        cudaStream_t stream) {
    return launch_chunk_impl<__nv_bfloat16, false>(plan, p, x, stream);
}

}  // namespace pkv
