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
// The tokens of one block stand behind one another in a call: a run, at most a block long.  A CTA
// has some heads of the runs that begin in a few rows of the call, a warp (two for pages of 32 x 128)
// the keys or values of one head: as many rows as a block has tokens are whole in its registers, 64
// numbers a lane at most, be they one run or many short ones.  It takes each run's largest |x|, then
// rounds.  Lane j looks after row j of that window: its slot, its run and that run's scale.  The warps of
// a CTA share the window's rows of the rotation table in shared memory.
#include <cfloat>
#include <type_traits>

#include "q8.cuh"
#include "rope.cuh"

namespace pkv {

namespace {

constexpr int Q8_Q_ROWS = 2;      // rows of q per group of lanes, in flight together
constexpr int Q8_KV_WARPS = 8;
// From this many tokens on q goes through rope_write.cu's kernels, a launch more.
constexpr int Q8_MANY_TOKENS = 512;
// Rows whose runs a CTA looks for.
constexpr int Q8_FEW_ROWS = 4, Q8_GROUP_ROWS = 16;
// What a scale reads as while the run that changes it is at work: a NaN that nothing else makes.
constexpr uint32_t Q8_LOCKED = 0xffc5a5c5u;

// A lane's part of a head row: where its two chunks lie, and whether they are rotated.
struct LanePart {
    int lo, hi, l;
    bool turns;
};

template <int P>
__device__ __forceinline__ void load_angles(const float* row, int R, int l, int V, float (&c)[2 * P], float (&s)[2 * P]) {
    row += l * (V / 2);
#pragma unroll
    for (int i = 0; i < 2 * P; i += 2) {
        const float2 x = *reinterpret_cast<const float2*>(row + i);
        const float2 y = *reinterpret_cast<const float2*>(row + R / 2 + i);
        c[i] = x.x; c[i + 1] = x.y;
        s[i] = y.x; s[i + 1] = y.y;
    }
}

// The q rows of token t, by the whole CTA.
template <typename T, int D, bool INTERLEAVED>
__device__ __forceinline__ void turn_queries(const RopeParams& p, const LanePart& at, int t) {
    constexpr int V = 8, LPR = D / V, P = 2;
    const int groups = blockDim.x / LPR, group = threadIdx.x / LPR, Hq = p.num_q_heads, R = p.rotary_dim;
    const int pos = p.positions[t];
    const long long slot = p.slot_mapping[t];
    if (pos < 0) return;  // a row that holds no token
    if (R > 0 && pos >= p.max_position) {
        if (threadIdx.x == 0) set_error(p.err, PKV_DEVERR_POSITION);
        return;
    }
    if (threadIdx.x == 0 && slot >= (long long)p.num_blocks * p.block_size) set_error(p.err, PKV_DEVERR_SLOT);
    float c[2 * P], s[2 * P];
    if (at.turns) load_angles<P>(p.cos_sin + (size_t)pos * R, R, at.l, V, c, s);
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
}

// Rounds a row of a page to a larger scale, a lane's 8 values.
__device__ __forceinline__ void round_again(uint2* at, float ratio) {
    const uint2 w = *at;
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
    *at = make_uint2(e4m3x4_of_floats(x[0], x[1], x[2], x[3]), e4m3x4_of_floats(x[4], x[5], x[6], x[7]));
}

}  // namespace

// The first q_ctas CTAs have the q rows of a token each; of the others, every `heads` have the runs that
// begin in `rows` rows.
template <typename T, int D, int B, bool INTERLEAVED>
__global__ void __launch_bounds__(Q8_KV_WARPS * 32, 2)
q8_write_kernel(const RopeParams p, float* k_scale, float* v_scale, int q_ctas, int heads, int rows) {
    constexpr int V = 8, LPR = D / V, P = 2;    // elements per lane, lanes per row
    constexpr int GPW = 32 / LPR;               // rows a warp at a time
    constexpr int W = B * D > 32 * 64 ? (B * D) / (16 * 128) : 1;  // warps a page
    constexpr int IT = B / (GPW * W);           // rows a lane
    static_assert(IT * 8 <= 64 && Q8_KV_WARPS % W == 0, "numbers a lane");
    __shared__ __align__(16) float angles[B * D];
    __shared__ float tops[Q8_KV_WARPS / W][32];
    __shared__ uint32_t hads[Q8_KV_WARPS / W][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int Hkv = p.num_kv_heads, R = p.rotary_dim;
    LanePart at;
    at.l = l;
    at.turns = l * V < R;
    at.lo = INTERLEAVED || !at.turns ? l * V : l * (V / 2);
    at.hi = INTERLEAVED || !at.turns ? at.lo + V / 2 : at.lo + R / 2;
    if ((int)blockIdx.x < q_ctas) {
        turn_queries<T, D, INTERLEAVED>(p, at, blockIdx.x);
        return;
    }
    const int cta = (int)blockIdx.x - q_ctas;
    const int u = cta % heads * (Q8_KV_WARPS / W) + warp / W, part = warp % W;
    const int first_u = u - warp / W;
    const bool real = u < 2 * Hkv, is_k = u < Hkv;
    const int head = real ? (is_k ? u : u - Hkv) : 0;
    const long long num_slots = (long long)p.num_blocks * B;
    const bool norm = p.k_weight != nullptr;
    float* const scales = is_k ? k_scale : v_scale;
    uint8_t* const pool = static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool);

    // slot and position of a row; slot -1: no key and value there
    auto look = [&](int i, int& pos) -> long long {
        pos = -1;
        if (i < 0 || i >= p.num_tokens) return -1;
        pos = p.positions[i];
        const long long slot = p.slot_mapping[i];
        return pos < 0 || (R > 0 && pos >= p.max_position) || slot < 0 || slot >= num_slots ? -1 : slot;
    };
    // A run: tokens whose slots advance as their rows do, in one block.  Row 0 of the window is t, lane j
    // has row j.
    const int t_end = min(cta / heads * rows + rows, p.num_tokens);
    bool first = true;
    for (int t = cta / heads * rows; t < t_end;) {
        int pos, unused;
        const long long slot = look(t + lane, pos);
        const long long blk = slot >= 0 ? slot / B : -1;
        const int row = (int)(slot - blk * B);
        const unsigned below = (1u << lane) - 1;
        const unsigned there = __ballot_sync(FULL_MASK, slot >= 0);
        // the nearest row before that holds a token: in the window, or (for its first token) before it
        int d = (there & below) != 0 ? lane - (31 - __clz(there & below)) : 0;
        long long other = __shfl_sync(FULL_MASK, slot, lane - d);
        if (first && there != 0) {
            const int j = __ffs(there) - 1;
            const long long before = look(t - 1 - lane, unused);
            const unsigned near = __ballot_sync(FULL_MASK, before >= 0);
            const long long nearest = __shfl_sync(FULL_MASK, before, near != 0 ? __ffs(near) - 1 : 0);
            if (lane == j && near != 0) {
                d = j + __ffs(near);
                other = nearest;
            }
        }
        const bool same = slot >= 0 && d > 0 && d <= max(row, 1) && other / B == blk;
        const bool follows = same && other == slot - d;
        const unsigned leaders = __ballot_sync(FULL_MASK, slot >= 0 && !follows);
        const unsigned refused = __ballot_sync(FULL_MASK, same && !follows);  // a slot twice, or in falling order
        // rows from the first leader on; those of a run that began before t are another CTA's
        const unsigned upto = leaders & (below | (1u << lane));
        const int lead = upto != 0 ? 31 - __clz(upto) : -1;
        const unsigned later = leaders & ~(below | (1u << lane));
        // where the row's run is known to end: before the next one, or with its block
        const int lead_row = __shfl_sync(FULL_MASK, row, max(lead, 0));
        const bool known = later != 0 || lead + B - lead_row <= 32;
        const bool member = slot >= 0 && lead >= 0;
        // runs that have a row past those held here, or may go on past the window, wait for the next one
        const unsigned over = __ballot_sync(FULL_MASK, member && (lane >= B || !known));
        const unsigned late = __ballot_sync(FULL_MASK, lead >= 0 && t + lead >= t_end);
        const int stop_over = over != 0 ? __shfl_sync(FULL_MASK, lead, __ffs(over) - 1) : 32;
        const int stop_late = late != 0 ? __ffs(late) - 1 : 32;
        const int stop = min(stop_over, stop_late);  // (a run that begins at row 0 is always whole)
        const unsigned run = __ballot_sync(FULL_MASK, member && lead < stop && !((refused >> max(lead, 0)) & 1));
        if (refused & ((stop < 32 ? 1u << stop : 0u) - 1) && threadIdx.x == 0) set_error(p.err, PKV_DEVERR_SLOT);
        const int t_now = t;
        t = stop < 32 ? t + stop : t + 32 > t_end ? t_end : t + 32;
        first = false;
        if (run == 0) continue;
        const int n = 32 - __clz(run);  // at most B
        const bool in_run = (run >> lane) & 1, leads = in_run && lead == lane;

        // the scale of each run's page, and no other run at that page from here on
        const size_t page = (size_t)max(blk, 0ll) * Hkv + head;
        uint32_t had = 0;
        if (real && leads && part == 0) had = atomicExch(reinterpret_cast<unsigned int*>(scales + page), Q8_LOCKED);

        // this lane's chunks of rows (part * IT + i) * GPW + sub
        uint2 a[IT], b[IT];
        const T* const base = (is_k ? static_cast<const T*>(p.k) + t_now * p.k_stride
                                    : static_cast<const T*>(p.v) + t_now * p.v_stride) + (size_t)head * D;
        const long long stride = is_k ? p.k_stride : p.v_stride;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = (part * IT + i) * GPW + sub;
            a[i] = b[i] = make_uint2(0u, 0u);
            if ((run >> r) & 1) {
                a[i] = __ldcs(reinterpret_cast<const uint2*>(base + r * stride + at.lo));
                b[i] = __ldcs(reinterpret_cast<const uint2*>(base + r * stride + at.hi));
            }
        }
        // the rows of the rotation table, for all warps
        if (R > 0 && first_u < Hkv) {
            for (int r = warp; r < n; r += Q8_KV_WARPS) {
                const int pr = __shfl_sync(FULL_MASK, pos, r);
                if ((run >> r) & 1)
                    for (int i = lane * 4; i < R; i += 128)
                        *reinterpret_cast<float4*>(angles + r * D + i) =
                            __ldg(reinterpret_cast<const float4*>(p.cos_sin + (size_t)pr * R + i));
            }
        }
        __syncthreads();

        float f[IT][8], most = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r0 = (part * IT + i) * GPW, r = r0 + sub;
            if (((run >> r0) & ((1u << GPW) - 1)) == 0) {  // the whole warp
#pragma unroll
                for (int k = 0; k < 8; ++k) f[i][k] = 0.f;
                continue;
            }
            uint64_t x[P], y[P];
            if (is_k) {
                float c[2 * P], s[2 * P];
                if (at.turns) load_angles<P>(angles + r * D, R, l, V, c, s);
                Turn<P> m;
                make_turn<T, INTERLEAVED, P>(m, p.k_weight, at.lo, at.hi, at.turns, c, s);
                turn_values<T, D, INTERLEAVED, P>(m, norm, at.turns, p.eps, a[i], b[i], x, y);
            } else {
                Chunk8<T>::unpack(a[i], x);
                Chunk8<T>::unpack(b[i], y);
            }
            unpack2(x[0], f[i][0], f[i][1]);
            unpack2(x[1], f[i][2], f[i][3]);
            unpack2(y[0], f[i][4], f[i][5]);
            unpack2(y[1], f[i][6], f[i][7]);
            if (!((run >> r) & 1)) {  // made from no angles
#pragma unroll
                for (int k = 0; k < 8; ++k) f[i][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(f[i][k]));  // (a NaN is left out)
        }
        if (__any_sync(FULL_MASK, most > FLT_MAX)) {  // infinities are left out too, and become NaN
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (!(fabsf(f[i][k]) <= FLT_MAX)) f[i][k] = __int_as_float(0x7fffffff);
        }
        // each row's largest, then each run's
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r0 = (part * IT + i) * GPW;
            if (((run >> r0) & ((1u << GPW) - 1)) == 0) continue;
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[i][k]));
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
            if (l == 0) tops[warp / W][r0 + sub] = m;
        }
        if constexpr (W > 1) {
            if (part == 0) hads[warp / W][lane] = had;
            __syncthreads();
            had = hads[warp / W][lane];
        } else {
            __syncwarp();
        }
        if (in_run) top = tops[warp / W][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float m = __shfl_up_sync(FULL_MASK, top, o);
            if (lane - o >= lead) top = fmaxf(top, m);  // (lead >= 0 where it matters)
        }
        top = __shfl_sync(FULL_MASK, top, later != 0 ? __ffs(later) - 2 : 31);
        had = __shfl_sync(FULL_MASK, had, max(lead, 0));
        const bool ok = real && in_run && had != Q8_LOCKED;
        if (real && in_run && !ok && leads) set_error(p.err, PKV_DEVERR_SLOT);
        const float old = __uint_as_float(had), need = q8_scale_for(top);
        const float s = lead_row > 0 ? fmaxf(old, need) : need;  // (a scale that is NaN counts as none)
        const float inv = 1.f / s, ratio = old / s;
        unsigned grown = __ballot_sync(FULL_MASK, ok && leads && lead_row > 0 && s > old);
        for (; grown != 0; grown &= grown - 1) {
            const int j = __ffs(grown) - 1, row0 = __shfl_sync(FULL_MASK, row, j);
            const unsigned rows_j = __ballot_sync(FULL_MASK, in_run && lead == j);
            const float ratio_j = __shfl_sync(FULL_MASK, ratio, j);
            uint8_t* const codes = pool + __shfl_sync(FULL_MASK, (unsigned long long)page, j) * (B * D);
            for (int r = part * GPW + sub; r < B; r += W * GPW) {
                const int k = j + r - row0;
                if (k < j || k > 31 || !((rows_j >> k) & 1))
                    round_again(reinterpret_cast<uint2*>(codes + r * D) + l, ratio_j);
            }
        }
        const unsigned stored = __ballot_sync(FULL_MASK, ok);
        const unsigned long long place = ((unsigned long long)page * B + row) * D;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r0 = (part * IT + i) * GPW, r = r0 + sub;
            if (((stored >> r0) & ((1u << GPW) - 1)) == 0) continue;
            const float by = __shfl_sync(FULL_MASK, inv, r);
            uint8_t* const out = pool + __shfl_sync(FULL_MASK, place, r);
            if ((stored >> r) & 1) {
                *reinterpret_cast<uint32_t*>(out + at.lo) =
                    e4m3x4_of_floats(f[i][0] * by, f[i][1] * by, f[i][2] * by, f[i][3] * by);
                *reinterpret_cast<uint32_t*>(out + at.hi) =
                    e4m3x4_of_floats(f[i][4] * by, f[i][5] * by, f[i][6] * by, f[i][7] * by);
            }
        }
        if (ok && leads && part == 0)
            atomicExch(reinterpret_cast<unsigned int*>(scales + page), __float_as_uint(s));
        __syncthreads();  // before the next window's rows of the table and maxima
    }
}

namespace {

template <typename T, int D, int B, bool INTERLEAVED>
cudaError_t launch_q8_write_tdbi(const RopeParams& p, float* k_scale, float* v_scale, cudaStream_t stream) {
    constexpr int W = B * D > 32 * 64 ? (B * D) / (16 * 128) : 1, UNITS = Q8_KV_WARPS / W;
    const long long heads = (2ll * p.num_kv_heads + UNITS - 1) / UNITS;
    const bool few = p.num_tokens < Q8_MANY_TOKENS;
    const int rows = few ? Q8_FEW_ROWS : Q8_GROUP_ROWS, q_ctas = few ? p.num_tokens : 0;
    const long long ctas = q_ctas + ((long long)p.num_tokens + rows - 1) / rows * heads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    q8_write_kernel<T, D, B, INTERLEAVED>
        <<<(unsigned)ctas, Q8_KV_WARPS * 32, 0, stream>>>(p, k_scale, v_scale, q_ctas, (int)heads, rows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || few) return e;
    RopeParams q = p;  // the q rows alone
    q.num_kv_heads = 0;
    return launch_rope_write(q, std::is_same<T, __half>::value ? PKV_F16 : PKV_BF16, stream);
}

template <typename T, int D>
cudaError_t launch_q8_write_td(const RopeParams& p, float* k_scale, float* v_scale, cudaStream_t stream) {
    if (p.block_size == 16)
        return p.interleaved ? launch_q8_write_tdbi<T, D, 16, true>(p, k_scale, v_scale, stream)
                             : launch_q8_write_tdbi<T, D, 16, false>(p, k_scale, v_scale, stream);
    return p.interleaved ? launch_q8_write_tdbi<T, D, 32, true>(p, k_scale, v_scale, stream)
                         : launch_q8_write_tdbi<T, D, 32, false>(p, k_scale, v_scale, stream);
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
