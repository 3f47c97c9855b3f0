// q8_decode_bf16.cu -- instantiates decode over 8-bit pools for __nv_bfloat16 queries.
#include "q8_decode.cuh"

namespace pkv {

template <>
cudaError_t launch_q8_decode<__nv_bfloat16>(const Q8DecodeParams& p, int head_dim, cudaStream_t stream) {
    return launch_q8_decode_impl<__nv_bfloat16>(p, head_dim, stream);
}

}  // namespace pkv
