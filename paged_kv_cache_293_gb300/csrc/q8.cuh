// q8.cuh -- the cache held in 8 bits: e4m3 values, a 32-bit scale per page (block and kv head).
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// Two e4m3 values (the low one first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    return h;
}
// Four e4m3 values of a word, as two pairs.
__device__ __forceinline__ void f16x4_of_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = f16x2_of_e4m3x2((uint16_t)w);
    hi = f16x2_of_e4m3x2((uint16_t)(w >> 16));
}
__device__ __forceinline__ float2 float2_of_f16x2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four values to the nearest e4m3, even at ties; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4_of_floats(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

constexpr int Q8_LEAST_POWER = -100;

// The least power of two, 2^-100 at least, whose 448 times reach x (finite, not negative): with
// x = f 2^e, 1 <= f < 2, that is 2^(e - 8) up to f = 1.75 = 448 / 256, and twice that above.
__device__ __forceinline__ float q8_scale_for(float x) {
    const int bits = __float_as_int(x);
    const int power = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return __int_as_float((max(power, Q8_LEAST_POWER) + 127) << 23);
}

// Decode over a pool held in 8 bits (q8_decode.cuh).
struct Q8DecodeParams {
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float* k_scale;
    const float* v_scale;
    int32_t num_blocks, block_size, num_kv_heads;
    const void* q;              // [S][NQ][Hq][D]
    int32_t num_seqs, num_queries, num_q_heads;
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t* context_lens;
    int32_t max_context_len;
    float scale_log2;           // scale * log2(e)
    int32_t partition_size, max_parts;
    int32_t column_tiles;       // columns (query, head) a CTA has, in tiles of 8: 1 or 2
    int32_t clustered;          // a context's pieces meet in a cluster's shared memory and not in the workspace
    void* out;
    int32_t out_dtype;
    float* part_m;              // base 2; [row][part], then sums, then [row][part][D]
    float* part_l;
    float* part_o;
    unsigned int* err;
};

// Pieces of a context up to which they are one cluster.
constexpr int Q8_CLUSTER = 8;
cudaError_t launch_q8_write(const RopeParams& p, float* k_scale, float* v_scale, int32_t dtype, cudaStream_t stream);
template <typename T>
cudaError_t launch_q8_decode(const Q8DecodeParams& p, int head_dim, cudaStream_t stream);
cudaError_t launch_q8_merge(const Q8DecodeParams& p, int head_dim, cudaStream_t stream);

}  // namespace pkv
