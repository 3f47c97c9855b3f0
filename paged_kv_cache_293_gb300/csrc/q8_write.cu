// q8_write.cu -- norms and rotation of queries and keys, and the keys and values into a cache
// held in 8 bits with a scale per page ("vLLM in Production", section "PagedAttention - Virtual
// Memory for the KV Cache": new tokens' keys and values enter the cache as they arrive).
//
// Rows are turned as in rope_write.cu.  A page (a block of tokens of one kv head) has one scale,
// a power of two s with 448 s >= |x| for all its numbers x, and holds e4m3(x / s).  e4m3's steps
// are relative (2^-4 of a value at most) down to 2^-6, so a power of two loses nothing against
// any other scale but where numbers are 2^-15 of the page's largest; and when a page that is
// partly filled needs a larger scale, its rows only change their exponents.
//
// The tokens of one block stand behind one another in a call.  The CTA of the first of such a run
// does all of it (a run is at most a block): a group of lanes has one kv head's keys or values,
// makes its rows once for their largest |x| and, where they are more than it holds, a second time
// to store them (their loads come from the L1 cache then).
#include <cfloat>

#include "q8.cuh"
#include "rope.cuh"

namespace pkv {

namespace {

constexpr int Q8_MAX_THREADS = 512;
constexpr int Q8_Q_ROWS = 2;    // rows of q per group of lanes, in flight together
constexpr int Q8_KV_ROWS = 4;   // rows of k or v
// What a scale reads as while the run that changes it is at work: a NaN that nothing else makes.
constexpr uint32_t Q8_LOCKED = 0xffc5a5c5u;

// A lane's part of a head row: where its two chunks lie, and whether they are rotated.
struct LanePart {
    int lo, hi, l;
    bool turns;
};

template <int P>
__device__ __forceinline__ void load_angles(const float* cos_sin, int pos, int R, int l, int V, float (&c)[2 * P],
                                            float (&s)[2 * P]) {
    const float* row = cos_sin + (size_t)pos * R + l * (V / 2);
#pragma unroll
    for (int i = 0; i < 2 * P; i += 2) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(row + i));
        const float2 y = __ldg(reinterpret_cast<const float2*>(row + R / 2 + i));
        c[i] = x.x; c[i + 1] = x.y;
        s[i] = y.x; s[i + 1] = y.y;
    }
}

// N rows of k (turned) or v (as they are) of one kv head, tokens t, t + 1, ...: this lane's eight
// numbers of each.  All lanes of the warp come here together; rows that are not of the run are
// made like the others and not used.
template <typename T, int D, bool INTERLEAVED, int N>
__device__ __forceinline__ void kv_rows(const RopeParams& p, const LanePart& at, bool is_k, int head, int t, int last,
                                        float (&f)[N][8]) {
    constexpr int V = 8, P = 2;
    uint2 a[N], b[N];
    int pos[N];
    const T* base = is_k ? static_cast<const T*>(p.k) : static_cast<const T*>(p.v);
    const long long stride = is_k ? p.k_stride : p.v_stride;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const int tr = min(t + r, last);
        const T* src = base + tr * stride + (size_t)head * D;
        a[r] = __ldg(reinterpret_cast<const uint2*>(src + at.lo));
        b[r] = __ldg(reinterpret_cast<const uint2*>(src + at.hi));
        pos[r] = min(max(p.positions[tr], 0), p.max_position - 1);
    }
#pragma unroll
    for (int r = 0; r < N; ++r) {
        float c[2 * P], s[2 * P];
        if (at.turns) load_angles<P>(p.cos_sin, pos[r], p.rotary_dim, at.l, V, c, s);
        Turn<P> m;
        make_turn<T, INTERLEAVED, P>(m, p.k_weight, at.lo, at.hi, at.turns, c, s);
        uint64_t x[P], y[P];
        turn_values<T, D, INTERLEAVED, P>(m, p.k_weight != nullptr, at.turns, p.eps, a[r], b[r], x, y);
        if (!is_k) {
            Chunk8<T>::unpack(a[r], x);
            Chunk8<T>::unpack(b[r], y);
        }
        unpack2(x[0], f[r][0], f[r][1]);
        unpack2(x[1], f[r][2], f[r][3]);
        unpack2(y[0], f[r][4], f[r][5]);
        unpack2(y[1], f[r][6], f[r][7]);
    }
}

template <int N>
__device__ __forceinline__ float largest_finite(const float (&f)[N][8], unsigned rows) {
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = fabsf(f[r][i]);
            if (((rows >> r) & 1) && x <= FLT_MAX) top = fmaxf(top, x);
        }
    return top;
}

template <int N>
__device__ __forceinline__ void store_rows(uint8_t* row, int D, const LanePart& at, const float (&f)[N][8],
                                           unsigned rows, float inv) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
        if (!((rows >> r) & 1)) continue;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (an infinity would become 448)
            x[i] = fabsf(f[r][i]) <= FLT_MAX ? f[r][i] * inv : __int_as_float(0x7fffffff);
        *reinterpret_cast<uint32_t*>(row + r * D + at.lo) = e4m3x4_of_floats(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint32_t*>(row + r * D + at.hi) = e4m3x4_of_floats(x[4], x[5], x[6], x[7]);
    }
}

}  // namespace

// blockIdx = (token, 0: its q rows, 1: the run of k and v rows that begins with it)
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(Q8_MAX_THREADS) q8_write_kernel(const RopeParams p, float* k_scale, float* v_scale) {
    constexpr int V = 8, LPR = D / V, P = 2;  // elements per lane, lanes per row
    const int t = blockIdx.x, groups = blockDim.x / LPR;
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR, lane = threadIdx.x & 31;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, R = p.rotary_dim, B = p.block_size;
    LanePart at;
    at.l = l;
    at.turns = l * V < R;
    at.lo = INTERLEAVED || !at.turns ? l * V : l * (V / 2);
    at.hi = INTERLEAVED || !at.turns ? at.lo + V / 2 : at.lo + R / 2;
    const long long num_slots = (long long)p.num_blocks * B;

    if (blockIdx.y == 0) {
        const int pos = p.positions[t];
        const long long slot = p.slot_mapping[t];
        if (pos < 0) return;  // a row that holds no token
        if (R > 0 && pos >= p.max_position) {
            if (threadIdx.x == 0) set_error(p.err, PKV_DEVERR_POSITION);
            return;
        }
        if (threadIdx.x == 0 && slot >= num_slots) set_error(p.err, PKV_DEVERR_SLOT);
        float c[2 * P], s[2 * P];
        if (at.turns) load_angles<P>(p.cos_sin, pos, R, l, V, c, s);
        Turn<P> m;
        make_turn<T, INTERLEAVED, P>(m, p.q_weight, at.lo, at.hi, at.turns, c, s);
        const T* src = static_cast<const T*>(p.q) + t * p.q_stride;
        T* dst = static_cast<T*>(p.q_out) + (size_t)t * Hq * D;
        for (int h0 = 0; h0 < Hq; h0 += groups * Q8_Q_ROWS) {
            uint2 a[Q8_Q_ROWS], b[Q8_Q_ROWS];
#pragma unroll
            for (int u = 0; u < Q8_Q_ROWS; ++u) {
                const int h = min(h0 + u * groups + group, Hq - 1);
                a[u] = __ldcs(reinterpret_cast<const uint2*>(src + h * D + at.lo));
                b[u] = __ldcs(reinterpret_cast<const uint2*>(src + h * D + at.hi));
            }
#pragma unroll
            for (int u = 0; u < Q8_Q_ROWS; ++u) {
                const int h = h0 + u * groups + group;
                turn_row<T, D, INTERLEAVED, P>(m, p.q_weight != nullptr, at.turns, p.eps, a[u], b[u]);
                if (h < Hq) {
                    *reinterpret_cast<uint2*>(dst + h * D + at.lo) = a[u];
                    *reinterpret_cast<uint2*>(dst + h * D + at.hi) = b[u];
                }
            }
        }
        return;
    }

    // ---- the run: of tokens whose slots advance as their rows do, in one block.  Lane i looks at
    // the i-th row from t on and the i-th before it.
    auto slot_of = [&](int i) -> long long {  // -1: no key and value there
        if (i < 0 || i >= p.num_tokens) return -1;
        const int pos = p.positions[i];
        const long long slot = p.slot_mapping[i];
        return pos < 0 || (R > 0 && pos >= p.max_position) || slot < 0 || slot >= num_slots ? -1 : slot;
    };
    const long long after = slot_of(t + lane), before = slot_of(t - 1 - lane);
    const long long slot = __shfl_sync(FULL_MASK, after, 0);
    if (slot < 0) return;
    const long long blk = slot / B;
    const int row0 = (int)(slot - blk * B);
    const unsigned near = __ballot_sync(FULL_MASK, before >= 0 && lane < max(row0, 1));
    if (near != 0) {  // the token before, where it may be of this block
        const int d = __ffs(near) - 1;
        const long long other = __shfl_sync(FULL_MASK, before, d);
        if (other / B == blk) {
            if (other != slot - 1 - d && threadIdx.x == 0) set_error(p.err, PKV_DEVERR_SLOT);
            return;  // in a run that an earlier token begins, or refused
        }
    }
    const unsigned fit = __ballot_sync(FULL_MASK, after == slot + lane && row0 + lane < B);
    const unsigned ends = __ballot_sync(FULL_MASK, after >= 0) & ~fit;  // bit 0 of fit is set
    const unsigned run = ends != 0 ? fit & ((ends & -ends) - 1) : fit;  // rows of the run, from t on
    const int n = 32 - __clz(run);

    for (int u0 = 0; u0 < 2 * Hkv; u0 += groups) {
        const int u = u0 + group;
        const bool real = u < 2 * Hkv, is_k = u < Hkv;
        if (!__any_sync(FULL_MASK, real)) break;
        const int head = real ? (is_k ? u : u - Hkv) : 0;
        const size_t page = (size_t)blk * Hkv + head;
        float* const scale = (is_k ? k_scale : v_scale) + page;
        uint8_t* const codes = static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool) + page * B * D;
        // the page's scale, and no other run at this page from here on
        uint32_t had = 0;
        if (real && l == 0) had = atomicExch(reinterpret_cast<unsigned int*>(scale), Q8_LOCKED);

        float f[Q8_KV_ROWS][8], top = 0.f;
        if (n == 1) {
            float one[1][8];
            kv_rows<T, D, INTERLEAVED, 1>(p, at, is_k, head, t, t, one);
            top = largest_finite<1>(one, 1u);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[0][i] = one[0][i];
        } else {
            for (int i = 0; i < n; i += Q8_KV_ROWS) {
                kv_rows<T, D, INTERLEAVED, Q8_KV_ROWS>(p, at, is_k, head, t + i, t + n - 1, f);
                top = fmaxf(top, largest_finite<Q8_KV_ROWS>(f, run >> i));
            }
        }
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        had = __shfl_sync(FULL_MASK, had, 0, LPR);
        const bool write = real && had != Q8_LOCKED;
        if (real && !write && l == 0) set_error(p.err, PKV_DEVERR_SLOT);
        const float old = __uint_as_float(had), need = q8_scale_for(top);
        const float s = row0 > 0 ? fmaxf(old, need) : need;  // (a scale that is NaN counts as none)
        if (write && row0 > 0 && s > old) {
            const float ratio = old / s;
            for (int r = 0; r < B; ++r) {
                if (r >= row0 && r < row0 + n && ((run >> (r - row0)) & 1)) continue;
                uint2* const at8 = reinterpret_cast<uint2*>(codes + r * D) + l;
                const uint2 w = *at8;
                uint32_t h[4];
                f16x4_of_e4m3x4(w.x, h[0], h[1]);
                f16x4_of_e4m3x4(w.y, h[2], h[3]);
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = float2_of_f16x2(h[i]);
                    x[2 * i] = v.x * ratio;
                    x[2 * i + 1] = v.y * ratio;
                }
                *at8 = make_uint2(e4m3x4_of_floats(x[0], x[1], x[2], x[3]), e4m3x4_of_floats(x[4], x[5], x[6], x[7]));
            }
        }
        const float inv = 1.f / s;
        uint8_t* const out = codes + row0 * D;
        if (n <= Q8_KV_ROWS) {
            if (write) store_rows<Q8_KV_ROWS>(out, D, at, f, run, inv);
        } else {
            for (int i = 0; i < n; i += Q8_KV_ROWS) {
                kv_rows<T, D, INTERLEAVED, Q8_KV_ROWS>(p, at, is_k, head, t + i, t + n - 1, f);
                if (write) store_rows<Q8_KV_ROWS>(out + i * D, D, at, f, run >> i, inv);
            }
        }
        if (write && l == 0) atomicExch(reinterpret_cast<unsigned int*>(scale), __float_as_uint(s));
    }
}

namespace {

template <typename T, int D>
cudaError_t launch_q8_write_td(const RopeParams& p, float* k_scale, float* v_scale, cudaStream_t stream) {
    constexpr int LPR = D / 8;
    const long long q_lanes = ((long long)p.num_q_heads + Q8_Q_ROWS - 1) / Q8_Q_ROWS * LPR;
    const long long kv_lanes = 2ll * p.num_kv_heads * LPR;
    const long long most = q_lanes > kv_lanes ? q_lanes : kv_lanes;
    const int threads = most >= Q8_MAX_THREADS ? Q8_MAX_THREADS : (int)((most + 31) / 32 * 32);
    const dim3 grid((unsigned)p.num_tokens, 2);
    if (p.interleaved)
        q8_write_kernel<T, D, true><<<grid, threads, 0, stream>>>(p, k_scale, v_scale);
    else
        q8_write_kernel<T, D, false><<<grid, threads, 0, stream>>>(p, k_scale, v_scale);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_q8_write_t(const RopeParams& p, float* k_scale, float* v_scale, cudaStream_t stream) {
    if (p.head_dim == 64) return launch_q8_write_td<T, 64>(p, k_scale, v_scale, stream);
    if (p.head_dim == 128) return launch_q8_write_td<T, 128>(p, k_scale, v_scale, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_q8_write(const RopeParams& p, float* k_scale, float* v_scale, int32_t dtype, cudaStream_t stream) {
    return dtype == PKV_F16 ? launch_q8_write_t<__half>(p, k_scale, v_scale, stream)
                            : launch_q8_write_t<__nv_bfloat16>(p, k_scale, v_scale, stream);
}

}  // namespace pkv
