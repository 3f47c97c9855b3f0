// q8_decode_f16.cu -- instantiates decode over 8-bit pools for __half queries, and the merge of
// contexts cut into pieces.
#include "q8_decode.cuh"

namespace pkv {

template <>
cudaError_t launch_q8_decode<__half>(const Q8DecodeParams& p, int head_dim, cudaStream_t stream) {
    return launch_q8_decode_impl<__half>(p, head_dim, stream);
}

// Row (s, j, h) of n > 1 pieces: M = max m_k, out = sum 2^(m_k - M) o_k / sum 2^(m_k - M) l_k.
// A CTA per row, warp w takes pieces w, w + warps, ... and a lane D / 32 elements.
constexpr int Q8_MERGE_WARPS = 16;

template <int D>
__global__ void __launch_bounds__(Q8_MERGE_WARPS * 32) q8_merge_kernel(const Q8DecodeParams p) {
    constexpr int V = D / 32;
    __shared__ float red[Q8_MERGE_WARPS][D + 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are the kernel before's
    const long long row = blockIdx.x;
    const int warps = blockDim.x / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (int)(row / ((long long)p.num_q_heads * p.num_queries));
    const long long table = (long long)p.max_blocks_per_seq * p.block_size;
    const int cap = (int)(table < p.max_context_len ? table : p.max_context_len);
    const int ctx = min(max(p.context_lens[s], 0), cap);
    const int n = (ctx + p.partition_size - 1) / p.partition_size;
    if (n <= 1) return;
    const float* m = p.part_m + (size_t)row * p.max_parts;
    const float* l = p.part_l + (size_t)row * p.max_parts;
    const float* o = p.part_o + (size_t)row * p.max_parts * D + lane * V;
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, m[k]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, d));
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[V] = {};
#pragma unroll 4
    for (int k = warp; k < n; k += warps) {
        const float by = fast_exp2(m[k] - ref);
        L = fmaf(by, l[k], L);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(by, o[(size_t)k * D + i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][lane * V + i] = acc[i];
    if (lane == 0) red[warp][D] = L;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float num = 0.f, den = 0.f;
        for (int w = 0; w < warps; ++w) {
            num += red[w][d];
            den += red[w][D];
        }
        // (-inf: a row that sees nothing)
        store_out(p.out, p.out_dtype, (size_t)row * D + d, M == -INFINITY ? 0.f : num / den);
    }
}

cudaError_t launch_q8_merge(const Q8DecodeParams& p, int head_dim, cudaStream_t stream) {
    const int warps = p.max_parts < 4 * Q8_MERGE_WARPS ? (p.max_parts + 3) / 4 : Q8_MERGE_WARPS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.num_seqs * p.num_queries * p.num_q_heads));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return head_dim == 64 ? cudaLaunchKernelEx(&cfg, q8_merge_kernel<64>, p)
                          : cudaLaunchKernelEx(&cfg, q8_merge_kernel<128>, p);
}

}  // namespace pkv
