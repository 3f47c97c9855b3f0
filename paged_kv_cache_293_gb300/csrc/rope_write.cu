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
// lane's rows, whose loads all start before anything waits; products run two to an
// instruction.
#include "pkv_common.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

// Rows per group of lanes, all in flight: few for few tokens, whose time is one row's way through
// the kernel (one token of 48 heads: 2.7 us with 2 rows, 4.3 us with 8; 128 tokens of 120 heads
// 3.2 and 4.1 us), more where the coefficients made per lane should serve several.
constexpr int ROPE_FEW_ROWS = 2, ROPE_ROWS = 8;
constexpr int ROPE_FEW_TOKENS = 512;
constexpr int ROPE_MAX_THREADS = 512;
constexpr int STREAM_MAX_STAGES = 4;
// Of stages per SM, at least three for each of four, two or one CTAs with four, eight or sixteen
// warps that turn rows; measured for the rows too wide for four CTAs, 4000 tokens: 40 + 2 * 40
// heads of 128, fp32 83.5 us (136 without streaming), 32 + 2 * 32 65.7 (86.3); 32 + 2 * 8, fp32
// 34.6 (36.4 with four warps in each of two CTAs), 64 + 2 * 8, bf16 35.1 (37.6).
constexpr int STREAM_BYTES = 216 * 1024;
// Streaming pays for its set-up and for its few instructions per copy from about this many
// values in all and bytes per token on; measured with head_dim 128, streaming against not:
// 32 + 2 * 8 heads, bf16: 512 tokens 4.9 / 5.0 us, 1024 7.0 / 9.2, 8192 36.1 / 58.0;
// 40 + 2 * 40, fp16: 256 tokens 6.4 / 5.2 us, 512 9.2 / 9.1, 8192 90.9 / 151.8;
// 16 + 2 * 4, fp32: 1024 tokens 6.3 / 5.2 us, 2048 8.7 / 8.6, 8192 35.5 / 42.9;
// rows of 3 KB (16 + 2 * 4 heads of 64, fp16): 8192 tokens 20.0 / 13.5 us.
constexpr long long STREAM_MIN_VALUES = 6 << 20;
constexpr long long STREAM_MIN_ROW = 6000;

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

// One row of q or k: both of this lane's chunks turned and scaled, in place.  The sum of
// squares takes all lanes of the warp.
template <typename T, int D, bool INTERLEAVED, int P>
__device__ __forceinline__ void turn_row(const Turn<P>& m, bool norm, bool turns, float eps, uint2& a2, uint2& b2) {
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
        float x, y;
        unpack2(sq, x, y);
        float ss = x + y;
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + eps);
        r2 = pack2(r, r);
    }
    uint64_t x[P], y[P];
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
    a2 = Chunk8<T>::pack(x);
    b2 = Chunk8<T>::pack(y);
}

}  // namespace

// FULL: every lane's elements are rotated (rotary_dim = D).
template <typename T, int D, bool INTERLEAVED, bool FULL, int ROWS>
__global__ void __launch_bounds__(ROPE_MAX_THREADS) rope_write_kernel(const RopeParams p) {
    constexpr int V = 16 / (int)sizeof(T);      // elements per lane
    constexpr int LPR = D / V;                  // lanes per row
    constexpr int P = Chunk8<T>::PAIRS;
    const int t = blockIdx.x, groups = blockDim.x / LPR;
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, H = Hq + 2 * Hkv;
    const int h0 = blockIdx.y * groups * ROWS + group;  // this group's first row, then every groups-th
    const int R = FULL ? D : p.rotary_dim, half = R / 2;
    // this lane's two chunks of a row: paired ones, or two in a row
    const bool turns = FULL || l * V < R;
    const int lo = INTERLEAVED || !turns ? l * V : l * (V / 2);
    const int hi = INTERLEAVED || !turns ? lo + V / 2 : lo + half;

    // every load that needs nothing else first: the rows, the position, the slot
    uint2 ra[ROWS], rb[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
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

    const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int h = h0 + u * groups;
        // the shuffles of a norm take whole warps: q and k rows of one warp go both ways
        const bool any_q = __any_sync(FULL_MASK, h < Hq), any_k = __any_sync(FULL_MASK, h >= Hq && h < Hq + Hkv);
        uint2 a = ra[u], b = rb[u];
        if (any_q) {
            turn_row<T, D, INTERLEAVED>(tq, norm_q, turns, p.eps, a, b);
            if (h < Hq) {
                T* dst = static_cast<T*>(p.q_out) + ((size_t)t * Hq + h) * D;
                *reinterpret_cast<uint2*>(dst + lo) = a;
                *reinterpret_cast<uint2*>(dst + hi) = b;
            }
        }
        if (any_k) {
            a = ra[u];
            b = rb[u];
            turn_row<T, D, INTERLEAVED>(tk, norm_k, turns, p.eps, a, b);
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

// Many tokens: CTAs that stay and stream them.  A token's q, k and v rows and its table row are
// each contiguous, so one thread brings them into a ring of stages by bulk copies; the other warps
// turn the q and k rows in place, and the same thread sends q out by one bulk copy and every
// head of k and v to its cache row by one each.  The copies keep running whatever the
// arithmetic does, which loads held in registers (rope_write_kernel) do not: 16384 tokens of
// 32 + 2 * 8 heads of 128 take 67 us here (411 MB, 6.1 TB/s) and 114 us there.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

template <typename T, int D, bool INTERLEAVED, bool FULL, int WARPS>
__global__ void __launch_bounds__((WARPS + 1) * 32) rope_stream_kernel(const RopeParams p, int stages,
                                                                     uint32_t stage_bytes) {
    constexpr int V = 16 / (int)sizeof(T), LPR = D / V, P = Chunk8<T>::PAIRS;
    constexpr int GROUPS = WARPS * 32 / LPR;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[2 * STREAM_MAX_STAGES];
    __shared__ int live[STREAM_MAX_STAGES];  // the stage holds a token
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, R = FULL ? D : p.rotary_dim, half = R / 2;
    const uint32_t q_bytes = (uint32_t)(Hq * D * (int)sizeof(T)), kv_bytes = (uint32_t)(Hkv * D * (int)sizeof(T));
    const int n = (p.num_tokens - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // tokens of this CTA
    const uint32_t bar0 = smem_addr(bars), ring0 = smem_addr(ring);
    auto full = [&](int st) { return bar0 + 8 * st; };
    auto done = [&](int st) { return bar0 + 8 * (STREAM_MAX_STAGES + st); };
    if (threadIdx.x == 0) {
        for (int st = 0; st < stages; ++st) {
            mbar_init(full(st), 1);
            mbar_init(done(st), WARPS);
        }
        mbar_init_fence();
    }
    __syncthreads();
    bool ok = true;
    if (warp == WARPS) {
        if (umma::elect_one()) {  // one thread as the compiler sees it: copies are issued faster
            const uint64_t policy = l2_evict_first_policy();  // the projections are not read again
            auto token = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };
            auto load = [&](int i, int pos) {
                const int st = i % stages;
                const long long t = token(i);
                const bool bad = R > 0 && pos >= p.max_position;
                if (bad) set_error(p.err, PKV_DEVERR_POSITION);
                live[st] = pos >= 0 && !bad;
                if (!live[st]) {
                    mbar_arrive(full(st));
                    return;
                }
                const uint32_t dst = ring0 + st * stage_bytes;
                mbar_arrive_expect_tx(full(st), q_bytes + 2 * kv_bytes + 4 * R);
                bulk_g2s(dst, static_cast<const T*>(p.q) + t * p.q_stride, q_bytes, full(st), policy);
                bulk_g2s(dst + q_bytes, static_cast<const T*>(p.k) + t * p.k_stride, kv_bytes, full(st), policy);
                bulk_g2s(dst + q_bytes + kv_bytes, static_cast<const T*>(p.v) + t * p.v_stride, kv_bytes, full(st),
                         policy);
                if (R > 0)
                    bulk_g2s(dst + q_bytes + 2 * kv_bytes, p.cos_sin + (size_t)pos * R, 4 * R, full(st), policy);
            };
            for (int i = 0; i < stages && i < n; ++i) load(i, p.positions[token(i)]);
            for (int i = 0; i < n; ++i) {
                const int st = i % stages, next = i - 1 + stages;
                const bool refill = i >= 1 && next < n;
                const int next_pos = refill ? p.positions[token(next)] : 0;
                long long slot = p.slot_mapping[token(i)];
                ok = mbar_wait_short(done(st), (i / stages) & 1);
                if (!ok) break;
                if (live[st]) {
                    const uint32_t src = ring0 + st * stage_bytes;
                    bulk_s2g(static_cast<T*>(p.q_out) + (size_t)token(i) * Hq * D, src, q_bytes);
                    if (slot >= (long long)p.num_blocks * p.block_size) {
                        set_error(p.err, PKV_DEVERR_SLOT);
                        slot = -1;
                    }
                    if (slot >= 0) {
                        const long long blk = slot / p.block_size;
                        const size_t row = ((size_t)blk * Hkv * p.block_size + (size_t)(slot - blk * p.block_size)) * D;
                        for (int h = 0; h < Hkv; ++h) {
                            const size_t at = row + (size_t)h * p.block_size * D;
                            const uint32_t k_src = src + q_bytes + h * (D * (uint32_t)sizeof(T));
                            bulk_s2g(static_cast<T*>(p.k_pool) + at, k_src, D * (uint32_t)sizeof(T));
                            bulk_s2g(static_cast<T*>(p.v_pool) + at, k_src + kv_bytes, D * (uint32_t)sizeof(T));
                        }
                    }
                }
                bulk_commit();
                if (refill) {  // the stage of the token before, once its copies out have read it
                    bulk_wait_read<1>();
                    load(next, next_pos);
                }
            }
            // the CTA must not end with copies still using its shared memory
            bulk_wait_read<0>();
            if (!ok)
                for (int st = 0; st < stages; ++st) mbar_wait_short(full(st), 0);
        }
    } else {
        const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
        const bool turns = FULL || l * V < R;
        const int lo = INTERLEAVED || !turns ? l * V : l * (V / 2);
        const int hi = INTERLEAVED || !turns ? lo + V / 2 : lo + half;
        const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
        // the groups with the fewest q rows take the first k rows
        const int first = (group + GROUPS - Hq % GROUPS) % GROUPS;
        for (int i = 0; i < n; ++i) {
            const int st = i % stages;
            ok = __all_sync(FULL_MASK, mbar_wait_short(full(st), (i / stages) & 1));
            if (!ok) break;
            if (live[st]) {
                unsigned char* stage = ring + (size_t)st * stage_bytes;
                float c[2 * P], s[2 * P];
                if (turns) {
                    const float* row = reinterpret_cast<const float*>(stage + q_bytes + 2 * kv_bytes) + l * (V / 2);
#pragma unroll
                    for (int x = 0; x < 2 * P; x += 2) {
                        const float2 cc = *reinterpret_cast<const float2*>(row + x);
                        const float2 sn = *reinterpret_cast<const float2*>(row + half + x);
                        c[x] = cc.x; c[x + 1] = cc.y;
                        s[x] = sn.x; s[x + 1] = sn.y;
                    }
                }
                // q rows, then k rows: whole warps take part in the sums
                Turn<P> m;
                make_turn<T, INTERLEAVED, P>(m, p.q_weight, lo, hi, turns, c, s);
                for (int h0 = 0; h0 < Hq; h0 += GROUPS) {
                    const int h = h0 + group;
                    T* row = reinterpret_cast<T*>(stage) + (size_t)(h < Hq ? h : 0) * D;
                    uint2 a = *reinterpret_cast<const uint2*>(row + lo), b = *reinterpret_cast<const uint2*>(row + hi);
                    turn_row<T, D, INTERLEAVED>(m, norm_q, turns, p.eps, a, b);
                    if (h < Hq) {
                        *reinterpret_cast<uint2*>(row + lo) = a;
                        *reinterpret_cast<uint2*>(row + hi) = b;
                    }
                }
                make_turn<T, INTERLEAVED, P>(m, p.k_weight, lo, hi, turns, c, s);
                for (int h0 = 0; h0 < Hkv; h0 += GROUPS) {
                    const int h = h0 + first;
                    if (!__any_sync(FULL_MASK, h < Hkv)) break;
                    T* row = reinterpret_cast<T*>(stage + q_bytes) + (size_t)(h < Hkv ? h : 0) * D;
                    uint2 a = *reinterpret_cast<const uint2*>(row + lo), b = *reinterpret_cast<const uint2*>(row + hi);
                    turn_row<T, D, INTERLEAVED>(m, norm_k, turns, p.eps, a, b);
                    if (h < Hkv) {
                        *reinterpret_cast<uint2*>(row + lo) = a;
                        *reinterpret_cast<uint2*>(row + hi) = b;
                    }
                }
                fence_proxy_async_shared();  // before the copies out, and the next copies in
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(done(st));
        }
    }
    if (!ok) set_error(p.err, PKV_DEVERR_TIMEOUT);
    __syncthreads();
}

namespace {

template <typename T, int D, bool INTERLEAVED, int ROWS>
cudaError_t launch_rope_rows(const RopeParams& p, cudaStream_t stream) {
    constexpr int LPR = D * (int)sizeof(T) / 16;
    const int H = p.num_q_heads + 2 * p.num_kv_heads;
    // one CTA holds all rows of a token where that takes at most ROPE_MAX_THREADS lanes, so the
    // token's table row is read by few; the lanes are whole warps
    const long long lanes = (long long)((H + ROWS - 1) / ROWS) * LPR;
    const long long ctas = (lanes + ROPE_MAX_THREADS - 1) / ROPE_MAX_THREADS;
    const long long threads = ((lanes + ctas - 1) / ctas + 31) / 32 * 32;
    const long long rows = threads / LPR * ROWS;
    if ((H + rows - 1) / rows > 65535) return cudaErrorInvalidConfiguration;
    dim3 grid(p.num_tokens, (unsigned)((H + rows - 1) / rows));
    if (p.rotary_dim == D)
        rope_write_kernel<T, D, INTERLEAVED, true, ROWS><<<grid, (unsigned)threads, 0, stream>>>(p);
    else
        rope_write_kernel<T, D, INTERLEAVED, false, ROWS><<<grid, (unsigned)threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int D, bool INTERLEAVED>
cudaError_t launch_rope_tdi(const RopeParams& p, cudaStream_t stream) {
    const int H = p.num_q_heads + 2 * p.num_kv_heads;
    const long long stage = ((long long)H * D * (int)sizeof(T) + 4ll * p.rotary_dim + 127) / 128 * 128;
    if (stage >= STREAM_MIN_ROW && 3 * stage <= STREAM_BYTES &&
        p.num_tokens * (stage / (int)sizeof(T)) >= STREAM_MIN_VALUES) {
        // (the wider ones ask for the rotated elements' number as they run)
        const int per_sm = 12 * stage <= STREAM_BYTES ? 4 : 6 * stage <= STREAM_BYTES ? 2 : 1;
        auto kernel = per_sm == 1   ? rope_stream_kernel<T, D, INTERLEAVED, false, 16>
                      : per_sm == 2 ? rope_stream_kernel<T, D, INTERLEAVED, false, 8>
                      : p.rotary_dim == D ? rope_stream_kernel<T, D, INTERLEAVED, true, 4>
                                          : rope_stream_kernel<T, D, INTERLEAVED, false, 4>;
        const int threads = (16 / per_sm + 1) * 32;
        const long long room = STREAM_BYTES / per_sm;
        const int stages = (int)(room / stage < STREAM_MAX_STAGES ? room / stage : STREAM_MAX_STAGES);
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, STREAM_BYTES);
        if (e != cudaSuccess) return e;
        const int ctas = p.num_tokens < sms * per_sm ? p.num_tokens : sms * per_sm;
        kernel<<<ctas, threads, (size_t)stages * stage, stream>>>(p, stages, (uint32_t)stage);
        return cudaGetLastError();
    }
    return p.num_tokens < ROPE_FEW_TOKENS ? launch_rope_rows<T, D, INTERLEAVED, ROPE_FEW_ROWS>(p, stream)
                                          : launch_rope_rows<T, D, INTERLEAVED, ROPE_ROWS>(p, stream);
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
