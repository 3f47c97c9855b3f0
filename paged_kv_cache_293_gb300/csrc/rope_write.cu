// rope_write.cu -- per-head norms of queries and keys, their rotation by position, and the
// keys and values into their cache slots, in one pass over the packed projection output
// ("vLLM in Production", section "PagedAttention - Virtual Memory for the KV Cache": new
// tokens' keys and values enter the cache as they arrive).
//
// For a head row x of D elements (32-bit throughout, one rounding at the end):
//   y = x / sqrt(mean(x^2) + eps) * w                     (left out without a weight)
//   (a, b) <- (a cos - b sin, b cos + a sin)              for each pair of the first R elements,
// pairs (i, i + R/2), or (2 i, 2 i + 1) when interleaved, with the cosines and sines of
// the token's position from a 32-bit table the caller makes (in 64 bits, so that far
// positions keep their angles).
//
// HBM bound: every row is read once and written once.  LPR lanes hold a row as 16-byte
// vectors, so the sum of squares is a butterfly over them and the other half of a rotated
// pair comes by a shuffle; a group of LPR lanes keeps its part of the token's table row in
// registers for all of its head rows and has ROPE_BATCH rows in flight.
#include "pkv_common.cuh"

namespace pkv {

namespace {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_BATCH = 4;  // rows in flight per group of lanes

template <typename T> struct PackOut;
template <> struct PackOut<float> {
    __device__ __forceinline__ static uint4 run(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <> struct PackOut<__half> {
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static uint4 run(const float* f) {
        return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
};
template <> struct PackOut<__nv_bfloat16> {
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static uint4 run(const float* f) {
        return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
};

}  // namespace

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(ROPE_THREADS) rope_write_kernel(const RopeParams p) {
    constexpr int V = 16 / (int)sizeof(T);      // elements per lane
    constexpr int LPR = D / V;                  // lanes per row
    constexpr int GROUPS = ROPE_THREADS / LPR;  // rows per step of the CTA
    constexpr int NC = INTERLEAVED ? V / 2 : V; // cosines per lane
    const int t = blockIdx.x;
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int pos = p.positions[t];
    if (pos < 0) return;  // a row that holds no token
    const int R = p.rotary_dim, half = R / 2;
    if (R > 0 && pos >= p.max_position) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_error(p.err, PKV_DEVERR_POSITION);
        return;
    }
    long long slot = p.slot_mapping[t];
    if (slot >= (long long)p.num_blocks * p.block_size) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_error(p.err, PKV_DEVERR_SLOT);
        slot = -1;
    }
    const long long blk = slot >= 0 ? slot / p.block_size : 0, in_blk = slot >= 0 ? slot % p.block_size : 0;

    // this lane's part of the table row: the same for every head of the token
    const int d0 = l * V;  // first element of this lane
    const bool turns = d0 < R;
    float c[NC], sn[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        c[i] = 1.f;
        sn[i] = 0.f;
    }
    if (turns) {
        const float* row = p.cos_sin + (size_t)pos * R;
        const int i0 = INTERLEAVED ? d0 / 2 : (d0 < half ? d0 : d0 - half);
        if constexpr (NC >= 4) {
#pragma unroll
            for (int i = 0; i < NC; i += 4) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
                const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
                c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
                sn[i] = b.x; sn[i + 1] = b.y; sn[i + 2] = b.z; sn[i + 3] = b.w;
            }
        } else {
            const float2 a = __ldg(reinterpret_cast<const float2*>(row + i0));
            const float2 b = __ldg(reinterpret_cast<const float2*>(row + half + i0));
            c[0] = a.x; c[1] = a.y;
            sn[0] = b.x; sn[1] = b.y;
        }
    }
    // the lane holding the other half of this lane's pairs, and the sign of its term
    const int lane = threadIdx.x & 31;
    const int partner = turns && !INTERLEAVED ? (d0 < half ? lane + half / V : lane - half / V) : lane;
    if (!INTERLEAVED && d0 < half) {
#pragma unroll
        for (int i = 0; i < NC; ++i) sn[i] = -sn[i];
    }

    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, H = Hq + 2 * Hkv;
    const int h_lo = (int)((long long)H * blockIdx.y / gridDim.y);
    const int h_hi = (int)((long long)H * (blockIdx.y + 1) / gridDim.y);
    for (int h0 = h_lo; h0 < h_hi; h0 += GROUPS * ROPE_BATCH) {
        uint4 raw[ROPE_BATCH];
#pragma unroll
        for (int u = 0; u < ROPE_BATCH; ++u) {
            const int h = h0 + u * GROUPS + group;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (h < h_hi) {
                const T* src = h < Hq ? static_cast<const T*>(p.q) + (long long)t * p.q_stride + (size_t)h * D
                               : h < Hq + Hkv
                                   ? static_cast<const T*>(p.k) + (long long)t * p.k_stride + (size_t)(h - Hq) * D
                                   : static_cast<const T*>(p.v) + (long long)t * p.v_stride + (size_t)(h - Hq - Hkv) * D;
                raw[u] = reinterpret_cast<const uint4*>(src)[l];
            }
        }
#pragma unroll
        for (int u = 0; u < ROPE_BATCH; ++u) {
            if (h0 + u * GROUPS >= h_hi) break;  // no group has a row (uniform over the CTA)
            const int h = h0 + u * GROUPS + group;
            float f[V];
            Elem<T>::to_float(raw[u], f);
            const void* w = h < Hq ? p.q_weight : p.k_weight;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
            if (w != nullptr) {
                float wf[V];
                Elem<T>::to_float(__ldg(reinterpret_cast<const uint4*>(w) + l), wf);
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = f[i] * r * wf[i];
            }
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float a = f[i], b = f[i + 1];
                    f[i] = turns ? a * c[i / 2] - b * sn[i / 2] : a;
                    f[i + 1] = turns ? b * c[i / 2] + a * sn[i / 2] : b;
                }
            } else {
                float other[V];
#pragma unroll
                for (int i = 0; i < V; ++i) other[i] = __shfl_sync(FULL_MASK, f[i], partner);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = turns ? f[i] * c[i] + other[i] * sn[i] : f[i];
            }
            if (h >= h_hi) continue;
            if (h < Hq) {
                T* dst = static_cast<T*>(p.q_out) + ((size_t)t * Hq + h) * D;
                reinterpret_cast<uint4*>(dst)[l] = PackOut<T>::run(f);
            } else if (slot >= 0) {
                const bool is_k = h < Hq + Hkv;
                const int kvh = is_k ? h - Hq : h - Hq - Hkv;
                T* pool = static_cast<T*>(is_k ? p.k_pool : p.v_pool);
                T* dst = pool + (((size_t)blk * Hkv + kvh) * p.block_size + in_blk) * D;
                reinterpret_cast<uint4*>(dst)[l] = is_k ? PackOut<T>::run(f) : raw[u];
            }
        }
    }
}

namespace {

template <typename T, int D>
cudaError_t launch_rope_td(const RopeParams& p, cudaStream_t stream) {
    constexpr int GROUPS = ROPE_THREADS / (D * (int)sizeof(T) / 16);
    const int H = p.num_q_heads + 2 * p.num_kv_heads;
    // few tokens: the heads of a token go to several CTAs of one batch of rows each
    const int steps = (H + GROUPS * ROPE_BATCH - 1) / (GROUPS * ROPE_BATCH);
    const int split = p.num_tokens < 1024 ? steps : 1;
    dim3 grid(p.num_tokens, split < 65535 ? split : 65535);
    if (p.interleaved)
        rope_write_kernel<T, D, true><<<grid, ROPE_THREADS, 0, stream>>>(p);
    else
        rope_write_kernel<T, D, false><<<grid, ROPE_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t stream) {
    if (p.head_dim == 64) return launch_rope_td<T, 64>(p, stream);
    if (p.head_dim == 128) return launch_rope_td<T, 128>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_write(const RopeParams& p, int32_t dtype, cudaStream_t stream) {
    switch (dtype) {
        case PKV_F32: return launch_rope_t<float>(p, stream);
        case PKV_F16: return launch_rope_t<__half>(p, stream);
        default: return launch_rope_t<__nv_bfloat16>(p, stream);
    }
}

}  // namespace pkv
