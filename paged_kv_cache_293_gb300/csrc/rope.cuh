// rope.cuh -- norm and rotation of one head row in registers, shared by the cache writes
// (rope_write.cu, q8_write.cu).
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// Bulk copies shared -> global, in groups; the wait for all but N groups to have read their bytes.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// V / 2 = 4 (16-bit) or 2 (32-bit) elements of 8 bytes, as pairs of 32-bit values and back.
template <typename T> struct Chunk8;
template <> struct Chunk8<float> {
    static constexpr int PAIRS = 1;
    __device__ __forceinline__ static void unpack(const uint2& r, uint64_t (&x)[1]) {
        x[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
    }
    __device__ __forceinline__ static uint2 pack(const uint64_t (&x)[1]) {
        float a, b;
        unpack2(x[0], a, b);
        return make_uint2(__float_as_uint(a), __float_as_uint(b));
    }
};
template <> struct Chunk8<__half> {
    static constexpr int PAIRS = 2;
    __device__ __forceinline__ static uint64_t up(uint32_t r) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
        return pack2(v.x, v.y);
    }
    __device__ __forceinline__ static uint32_t down(uint64_t x) {
        float a, b;
        unpack2(x, a, b);
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static void unpack(const uint2& r, uint64_t (&x)[2]) {
        x[0] = up(r.x);
        x[1] = up(r.y);
    }
    __device__ __forceinline__ static uint2 pack(const uint64_t (&x)[2]) {
        return make_uint2(down(x[0]), down(x[1]));
    }
};
template <> struct Chunk8<__nv_bfloat16> {
    static constexpr int PAIRS = 2;
    __device__ __forceinline__ static uint64_t up(uint32_t r) {
        return pack2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t down(uint64_t x) {
        float a, b;
        unpack2(x, a, b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static void unpack(const uint2& r, uint64_t (&x)[2]) {
        x[0] = up(r.x);
        x[1] = up(r.y);
    }
    __device__ __forceinline__ static uint2 pack(const uint64_t (&x)[2]) {
        return make_uint2(down(x[0]), down(x[1]));
    }
};

__device__ __forceinline__ uint64_t swap2(uint64_t x) {
    float a, b;
    unpack2(x, a, b);
    return pack2(b, a);
}

// What a lane multiplies its two chunks a and b with, for one weight vector.
//   halves paired:  a <- a aa + b ab,  b <- b bb + a ba
//   interleaved:    a <- a aa + swap(a) ab,  b <- b bb + swap(b) ba
template <int P>
struct Turn {
    uint64_t aa[P], ab[P], bb[P], ba[P];
};

template <typename T, bool INTERLEAVED, int P>
__device__ __forceinline__ void make_turn(Turn<P>& m, const void* w, int lo, int hi, bool turns,
                                          const float* c, const float* s) {
    uint64_t wa[P], wb[P];
#pragma unroll
    for (int i = 0; i < P; ++i) wa[i] = wb[i] = pack2(1.f, 1.f);
    if (w != nullptr) {
        Chunk8<T>::unpack(__ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + lo)), wa);
        Chunk8<T>::unpack(__ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + hi)), wb);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (!turns) {
            m.aa[i] = wa[i];
            m.bb[i] = wb[i];
            m.ab[i] = m.ba[i] = 0;
        } else if (INTERLEAVED) {
            // pair i of a turns by c[i], pair i of b by c[P + i]
            m.aa[i] = mul2(wa[i], pack2(c[i], c[i]));
            m.ab[i] = mul2(swap2(wa[i]), pack2(-s[i], s[i]));
            m.bb[i] = mul2(wb[i], pack2(c[P + i], c[P + i]));
            m.ba[i] = mul2(swap2(wb[i]), pack2(-s[P + i], s[P + i]));
        } else {
            m.aa[i] = mul2(wa[i], pack2(c[2 * i], c[2 * i + 1]));
            m.ab[i] = mul2(wb[i], pack2(-s[2 * i], -s[2 * i + 1]));
            m.bb[i] = mul2(wb[i], pack2(c[2 * i], c[2 * i + 1]));
            m.ba[i] = mul2(wa[i], pack2(s[2 * i], s[2 * i + 1]));
        }
    }
}

// One row of q or k: both of this lane's chunks turned and scaled, as 32-bit values.  The sum of
// squares takes all lanes of the warp.
template <typename T, int D, bool INTERLEAVED, int P>
__device__ __forceinline__ void turn_values(const Turn<P>& m, bool norm, bool turns, float eps, const uint2& a2,
                                            const uint2& b2, uint64_t (&x)[P], uint64_t (&y)[P]) {
    constexpr int LPR = D * (int)sizeof(T) / 16;
    uint64_t a[P], b[P];
    Chunk8<T>::unpack(a2, a);
    Chunk8<T>::unpack(b2, b);
    uint64_t r2 = 0;
    if (norm) {
        uint64_t sq = mul2(a[0], a[0]);
        sq = fma2(b[0], b[0], sq);
#pragma unroll
        for (int i = 1; i < P; ++i) {
            sq = fma2(a[i], a[i], sq);
            sq = fma2(b[i], b[i], sq);
        }
        float u, v;
        unpack2(sq, u, v);
        float ss = u + v;
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + eps);
        r2 = pack2(r, r);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        x[i] = mul2(a[i], m.aa[i]);
        y[i] = mul2(b[i], m.bb[i]);
        if (turns) {  // elements past the rotated ones meet no zero factor
            x[i] = fma2(INTERLEAVED ? swap2(a[i]) : b[i], m.ab[i], x[i]);
            y[i] = fma2(INTERLEAVED ? swap2(b[i]) : a[i], m.ba[i], y[i]);
        }
        if (norm) {
            x[i] = mul2(x[i], r2);
            y[i] = mul2(y[i], r2);
        }
    }
}

// The same in place, rounded to the row's type.
template <typename T, int D, bool INTERLEAVED, int P>
__device__ __forceinline__ void turn_row(const Turn<P>& m, bool norm, bool turns, float eps, uint2& a2, uint2& b2) {
    uint64_t x[P], y[P];
    turn_values<T, D, INTERLEAVED, P>(m, norm, turns, eps, a2, b2, x, y);
    a2 = Chunk8<T>::pack(x);
    b2 = Chunk8<T>::pack(y);
}

}  // namespace pkv
