// chunk_q8_bf16.cu -- instantiates the chunk attention kernel for __nv_bfloat16 queries over 8-bit pools.
#include "chunk.cuh"

namespace pkv {

template <>
cudaError_t launch_chunk_q8<__nv_bfloat16>(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                                cudaStream_t stream) {
    return launch_chunk_impl<__nv_bfloat16, true>(plan, p, x, stream);
}

}  // namespace pkv
