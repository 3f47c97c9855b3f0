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
// HBM bound (every row is read once and written once) as long as the arithmetic stays out of
// the way, so it is laid out to need few instructions: LPR lanes hold a row, a lane both
// elements of each of its pairs (8 bytes of the first half and 8 of the second when the
// halves are paired), so nothing but the sum of squares crosses lanes; weight times cosine and
// weight times sine are made once per token and lane, for q and for k, and serve all of the
// lane's ROPE_ROWS rows, whose loads all start before anything waits; products run two to an
// instruction.
#include "pkv_common.cuh"

namespace pkv {

namespace {

constexpr int ROPE_ROWS = 8;           // rows per group of lanes, all in flight
constexpr int ROPE_MAX_THREADS = 512;

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

}  // namespace

// FULL: every lane's elements are rotated (rotary_dim = D).
template <typename T, int D, bool INTERLEAVED, bool FULL>
__global__ void __launch_bounds__(ROPE_MAX_THREADS) rope_write_kernel(const RopeParams p) {
    constexpr int V = 16 / (int)sizeof(T);      // elements per lane
    constexpr int LPR = D / V;                  // lanes per row
    constexpr int P = Chunk8<T>::PAIRS;
    const int t = blockIdx.x, groups = blockDim.x / LPR;
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, H = Hq + 2 * Hkv;
    const int h0 = blockIdx.y * groups * ROPE_ROWS + group;  // this group's first row, then every groups-th
    const int R = FULL ? D : p.rotary_dim, half = R / 2;
    // this lane's two chunks of a row: paired ones, or two in a row
    const bool turns = FULL || l * V < R;
    const int lo = INTERLEAVED || !turns ? l * V : l * (V / 2);
    const int hi = INTERLEAVED || !turns ? lo + V / 2 : lo + half;

    // every load that needs nothing else first: the rows, the position, the slot
    uint2 ra[ROPE_ROWS], rb[ROPE_ROWS];
#pragma unroll
    for (int u = 0; u < ROPE_ROWS; ++u) {
        const int h = h0 + u * groups;
        ra[u] = rb[u] = make_uint2(0u, 0u);
        if (h < H) {
            const T* src = h < Hq ? static_cast<const T*>(p.q) + (long long)t * p.q_stride + (size_t)h * D
                           : h < Hq + Hkv
                               ? static_cast<const T*>(p.k) + (long long)t * p.k_stride + (size_t)(h - Hq) * D
                               : static_cast<const T*>(p.v) + (long long)t * p.v_stride + (size_t)(h - Hq - Hkv) * D;
            ra[u] = __ldcs(reinterpret_cast<const uint2*>(src + lo));
            rb[u] = __ldcs(reinterpret_cast<const uint2*>(src + hi));
        }
    }
    const int pos = p.positions[t];
    long long slot = p.slot_mapping[t];
    if (pos < 0) return;  // a row that holds no token
    const bool reports = threadIdx.x == 0 && blockIdx.y == 0;
    if (R > 0 && pos >= p.max_position) {
        if (reports) set_error(p.err, PKV_DEVERR_POSITION);
        return;
    }
    if (slot >= (long long)p.num_blocks * p.block_size) {
        if (reports) set_error(p.err, PKV_DEVERR_SLOT);
        slot = -1;
    }
    float c[2 * P], s[2 * P];
    if (turns) {
        const float* row = p.cos_sin + (size_t)pos * R + l * (V / 2);
#pragma unroll
        for (int i = 0; i < 2 * P; i += 2) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(row + i));
            const float2 y = __ldg(reinterpret_cast<const float2*>(row + half + i));
            c[i] = x.x; c[i + 1] = x.y;
            s[i] = y.x; s[i + 1] = y.y;
        }
    }
    Turn<P> tq, tk;
    make_turn<T, INTERLEAVED, P>(tq, p.q_weight, lo, hi, turns, c, s);
    make_turn<T, INTERLEAVED, P>(tk, p.k_weight, lo, hi, turns, c, s);
    const long long blk = slot >= 0 ? slot / p.block_size : 0;
    const int in_blk = (int)(slot - blk * p.block_size);
    const size_t kv_row = ((size_t)blk * Hkv * p.block_size + in_blk) * D;  // of kv head 0

    // one row of q or k: both chunks turned and scaled, in place
    auto turn_row = [&](const Turn<P>& m, bool norm, uint2& a2, uint2& b2) {
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
            float x, y;
            unpack2(sq, x, y);
            float ss = x + y;
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            r2 = pack2(r, r);
        }
        uint64_t x[P], y[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            x[i] = mul2(a[i], m.aa[i]);
            y[i] = mul2(b[i], m.bb[i]);
            if (FULL || turns) {  // elements past the rotated ones meet no zero factor
                x[i] = fma2(INTERLEAVED ? swap2(a[i]) : b[i], m.ab[i], x[i]);
                y[i] = fma2(INTERLEAVED ? swap2(b[i]) : a[i], m.ba[i], y[i]);
            }
            if (norm) {
                x[i] = mul2(x[i], r2);
                y[i] = mul2(y[i], r2);
            }
        }
        a2 = Chunk8<T>::pack(x);
        b2 = Chunk8<T>::pack(y);
    };
    const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
#pragma unroll
    for (int u = 0; u < ROPE_ROWS; ++u) {
        const int h = h0 + u * groups;
        // the shuffles of a norm take whole warps: q and k rows of one warp go both ways
        const bool any_q = __any_sync(FULL_MASK, h < Hq), any_k = __any_sync(FULL_MASK, h >= Hq && h < Hq + Hkv);
        uint2 a = ra[u], b = rb[u];
        if (any_q) {
            turn_row(tq, norm_q, a, b);
            if (h < Hq) {
                T* dst = static_cast<T*>(p.q_out) + ((size_t)t * Hq + h) * D;
                *reinterpret_cast<uint2*>(dst + lo) = a;
                *reinterpret_cast<uint2*>(dst + hi) = b;
            }
        }
        if (any_k) {
            a = ra[u];
            b = rb[u];
            turn_row(tk, norm_k, a, b);
        }
        if (h >= Hq && h < H && slot >= 0) {
            const bool is_k = h < Hq + Hkv;
            T* dst = static_cast<T*>(is_k ? p.k_pool : p.v_pool) + kv_row +
                     (size_t)(is_k ? h - Hq : h - Hq - Hkv) * p.block_size * D;
            *reinterpret_cast<uint2*>(dst + lo) = is_k ? a : ra[u];
            *reinterpret_cast<uint2*>(dst + hi) = is_k ? b : rb[u];
        }
    }
}

namespace {

template <typename T, int D, bool INTERLEAVED>
cudaError_t launch_rope_tdi(const RopeParams& p, cudaStream_t stream) {
    constexpr int LPR = D * (int)sizeof(T) / 16;
    const int H = p.num_q_heads + 2 * p.num_kv_heads;
    // one CTA holds all rows of a token where that takes at most ROPE_MAX_THREADS lanes, so the
    // token's table row is read by few; the lanes are whole warps
    const long long lanes = (long long)((H + ROPE_ROWS - 1) / ROPE_ROWS) * LPR;
    const long long ctas = (lanes + ROPE_MAX_THREADS - 1) / ROPE_MAX_THREADS;
    const long long threads = ((lanes + ctas - 1) / ctas + 31) / 32 * 32;
    const long long rows = threads / LPR * ROPE_ROWS;
    if ((H + rows - 1) / rows > 65535) return cudaErrorInvalidConfiguration;
    dim3 grid(p.num_tokens, (unsigned)((H + rows - 1) / rows));
    if (p.rotary_dim == D)
        rope_write_kernel<T, D, INTERLEAVED, true><<<grid, (unsigned)threads, 0, stream>>>(p);
    else
        rope_write_kernel<T, D, INTERLEAVED, false><<<grid, (unsigned)threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rope_td(const RopeParams& p, cudaStream_t stream) {
    return p.interleaved ? launch_rope_tdi<T, D, true>(p, stream) : launch_rope_tdi<T, D, false>(p, stream);
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
