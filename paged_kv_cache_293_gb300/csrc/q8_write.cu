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
// The tokens of one block stand behind one another in a call: a run, at most a block long.  A window is
// as many rows of the call as a block has tokens: one run or several short ones, whole.  A warp (two
// for pages of 32 x 128) has the keys or values of one head of a window in its registers, 64 numbers a
// lane at most: it takes each run's largest |x|, then rounds.  Lane j looks after row j: its slot, its
// run and that run's scale.
// Measured: one token of 32 + 2 * 8 heads of 128 4.9 us (two dependent round trips to memory, the slots and
// then rows, scales and table), 128 of 40 + 2 * 40 7.7; 16384 of 32 + 2 * 8, bf16, 76 us (378 MB, 5.0 TB/s);
// q alone, through rope_write.cu, takes 50 of them, and the keys and values 28: about 6000 cycles a window
// of 16 tokens and CTA, bound by instructions (46 % of the issue slots) at 16 warps per SM, whose numbers
// take all registers.
#include <cfloat>
#include <type_traits>

#include "decode_mma.cuh"
#include "q8.cuh"
#include "rope.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr int Q8_Q_ROWS = 2;      // rows of q per group of lanes, in flight together
constexpr int Q8_KV_WARPS = 8;
// From this many tokens on q goes through rope_write.cu's kernels and k and v are streamed by a second launch.
// One launch against these two, one after the other, bf16:
//   32 + 2 * 8 heads of 128    1024 tokens 12.3 / 13.0 us    2048 tokens 20.4 / 18.6
//   40 + 2 * 40 heads of 128   1024 tokens 23.2 / 24.6       1536 tokens 33.6 / 28.7
//   16 + 2 * 4 heads of 64     1024 tokens 10.8 / 10.9       2048 tokens 15.0 / 10.9
// The second launch begins where the first leaves room: 2048 tokens of 32 + 2 * 8 heads 17.1 us (18.8 one after
// the other), 16384 76 (79.5); 2048 decoding requests of 40 + 2 * 40 heads 43.5 (42.4).
constexpr int Q8_MANY_TOKENS = 1025;
// Rows whose runs a CTA looks for: few while that makes no more CTAs of keys and values than fit the SMs at a
// time, two each.  Decoding requests, 4 rows / 16 rows:
//   32 + 2 * 8 heads of 128    16 requests 5.3 / 6.2 us    256 requests 7.6 / 6.9    384 8.5 / 9.6 (4 rows taken)
//   40 + 2 * 40 heads of 128   64 requests 6.7 / 6.9       128 requests 9.9 / 8.0    512 28.0 / 15.7 (16 from 122 on)
// (Counted with q's CTAs, it would gain 0.7 us at the 256 and lose 1.1 at the 384.)
constexpr int Q8_CTAS_PER_SM = 2;
constexpr int Q8_FEW_ROWS = 4, Q8_GROUP_ROWS = 16;
// What a scale reads as while the run that changes it is at work: a NaN that nothing else makes.
constexpr uint32_t Q8_LOCKED = 0xffc5a5c5u;

// A lane's part of a head row: where its two chunks lie, and whether they are rotated.
struct LanePart {
    int lo, hi, l;
    bool turns;
};

__device__ __forceinline__ void load_angles(const float* row, int R, int l, float (&c)[4], float (&s)[4]) {
    const float4 x = *reinterpret_cast<const float4*>(row + l * 4);
    const float4 y = *reinterpret_cast<const float4*>(row + R / 2 + l * 4);
    c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
    s[0] = y.x; s[1] = y.y; s[2] = y.z; s[3] = y.w;
}

// The q rows of token t, by the whole CTA.
template <typename T, int D, bool INTERLEAVED>
__device__ __forceinline__ void turn_queries(const RopeParams& p, const LanePart& at, int t) {
    constexpr int LPR = D / 8, P = 2;
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
    if (at.turns) load_angles(p.cos_sin + (size_t)pos * R, R, at.l, c, s);
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

// Which lanes rotate their part of a row.
enum class Turning { NONE, SOME, ALL };

// A lane's chunks a and b of a key, times the weights wa and wb (ones: without a norm) and turned by the
// table's row; by: the factor that the norm asks for besides.  No branches, so that several rows' chains
// run side by side.  All lanes of the warp.
template <typename T, int D, bool INTERLEAVED, Turning TURN>
__device__ __forceinline__ void make_key(const uint2& a2, const uint2& b2, const float* angles, int R, bool norm,
                                         const uint64_t (&wa)[2], const uint64_t (&wb)[2], const LanePart& at, float eps,
                                         uint64_t (&f)[4], float& by) {
    uint64_t x[2], y[2];
    Chunk8<T>::unpack(a2, x);
    Chunk8<T>::unpack(b2, y);
    float u, v;
    unpack2(fma2(y[1], y[1], fma2(x[1], x[1], fma2(y[0], y[0], mul2(x[0], x[0])))), u, v);
    float ss = u + v;
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + eps);
    by = norm ? r : 1.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[i] = mul2(x[i], wa[i]);
        y[i] = mul2(y[i], wb[i]);
    }
    f[0] = x[0];
    f[1] = x[1];
    f[2] = y[0];
    f[3] = y[1];
    if constexpr (TURN != Turning::NONE) {
        float c[4], s[4];
        load_angles(angles, R, at.l, c, s);  // (a lane that does not turn: its share of whatever lies there)
        uint64_t g[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (INTERLEAVED) {  // pair i of a turns by c[i], pair i of b by c[2 + i]
                g[i] = fma2(swap2(x[i]), pack2(-s[i], s[i]), mul2(x[i], pack2(c[i], c[i])));
                g[2 + i] = fma2(swap2(y[i]), pack2(-s[2 + i], s[2 + i]), mul2(y[i], pack2(c[2 + i], c[2 + i])));
            } else {
                const uint64_t cc = pack2(c[2 * i], c[2 * i + 1]);
                g[i] = fma2(y[i], pack2(-s[2 * i], -s[2 * i + 1]), mul2(x[i], cc));
                g[2 + i] = fma2(x[i], pack2(s[2 * i], s[2 * i + 1]), mul2(y[i], cc));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = TURN == Turning::ALL || at.turns ? g[i] : f[i];
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

// What lane j knows of row j of a window that begins at row t of the call.
struct Window {
    int blk, row, pos;    // block (-1: no key and value there), place in it, position
    int lead, last;       // the first and the last row of its run
    int lead_row;         // the first one's place in the block
    unsigned run;         // all lanes: the rows that are written, and those that begin a run
    unsigned leaders;
};

// A row's slot and position as the call has them (none past its rows).
struct RawRow {
    long long slot;
    int pos;
};
__device__ __forceinline__ RawRow load_row(const RopeParams& p, int i) {
    if (i < 0 || i >= p.num_tokens) return RawRow{-1, -1};
    return RawRow{p.slot_mapping[i], p.positions[i]};
}

// The block that a row's token lies in (-1: there is none) and its place there.
template <int B>
__device__ __forceinline__ int block_of(const RopeParams& p, const RawRow& x, int& row) {
    row = -1;
    if (x.pos < 0 || (p.rotary_dim > 0 && x.pos >= p.max_position) || x.slot < 0 ||
        x.slot >= (long long)p.num_blocks * B)
        return -1;
    row = (int)(x.slot & (B - 1));
    return (int)(x.slot / B);
}

// The nearest row with a token before a window (blk: -1 where none of the 32 rows before has one).
struct Before {
    int blk, row, at;
};
template <int B>
__device__ __forceinline__ Before before_row(const RopeParams& p, int t) {
    int row;
    const int blk = block_of<B>(p, load_row(p, t - 1 - (int)(threadIdx.x & 31)), row);
    const unsigned near = __ballot_sync(FULL_MASK, blk >= 0);
    const int k = near != 0 ? __ffs(near) - 1 : 0;
    return Before{__shfl_sync(FULL_MASK, blk, k), __shfl_sync(FULL_MASK, row, k), t - 1 - k};
}

// The runs that begin in rows [t, t_end) and are whole in the B rows from t on; t moves to the first that
// is not, and `before` with it.  A run: tokens whose slots advance as their rows do, in one block.  raw:
// lane j's row t + j.  Whole warps.
template <int B>
__device__ __forceinline__ Window find_window(const RopeParams& p, const RawRow& raw, Before& before, int& t,
                                              int t_end, bool reports) {
    const int lane = threadIdx.x & 31;
    Window w;
    w.pos = raw.pos;
    w.blk = block_of<B>(p, raw, w.row);
    const unsigned below = (1u << lane) - 1, here = 1u << lane;
    const unsigned there = __ballot_sync(FULL_MASK, w.blk >= 0);
    // the nearest row before that holds a token: in the window, or (for its first token) before it
    int d = (there & below) != 0 ? lane - (31 - __clz(there & below)) : 0;
    int blk_d = __shfl_sync(FULL_MASK, w.blk, lane - d), row_d = __shfl_sync(FULL_MASK, w.row, lane - d);
    if (lane == __ffs(there) - 1 && before.blk >= 0) {
        d = t + lane - before.at;
        blk_d = before.blk;
        row_d = before.row;
    }
    const bool same = w.blk >= 0 && d > 0 && d <= 32 && blk_d == w.blk;
    const bool follows = same && row_d == w.row - d;
    w.leaders = __ballot_sync(FULL_MASK, w.blk >= 0 && !follows);
    const unsigned refused = __ballot_sync(FULL_MASK, same && !follows);  // a slot twice, or in falling order
    // (rows before the first leader are of a run that began before t, another CTA's)
    const unsigned upto = w.leaders & (below | here), later = w.leaders & ~(below | here);
    const int lead = upto != 0 ? 31 - __clz(upto) : -1;
    w.lead = max(lead, 0);
    w.last = later != 0 ? __ffs(later) - 2 : 31;
    w.lead_row = __shfl_sync(FULL_MASK, w.row, w.lead);
    // where the row's run is known to end: before the next one, or with its block
    const bool known = later != 0 || lead + B - w.lead_row <= 32;
    const bool member = w.blk >= 0 && lead >= 0;
    // runs that have a row past those held here, or may go on past the window, wait for the next one
    // (a run that begins at row 0 is always whole)
    const unsigned over = __ballot_sync(FULL_MASK, member && (lane >= B || !known));
    const unsigned late = __ballot_sync(FULL_MASK, lead >= 0 && t + lead >= t_end);
    const int stop_over = over != 0 ? __shfl_sync(FULL_MASK, lead, __ffs(over) - 1) : 32;
    const int stop = min(stop_over, late != 0 ? __ffs(late) - 1 : 32);
    w.run = __ballot_sync(FULL_MASK, member && lead < stop && !((refused >> w.lead) & 1));
    if (reports && (refused & ((stop < 32 ? 1u << stop : 0u) - 1)) != 0) set_error(p.err, PKV_DEVERR_SLOT);
    const unsigned passed = there & (stop < 32 ? (1u << stop) - 1 : FULL_MASK);
    if (passed != 0) {
        const int k = 31 - __clz(passed);
        before = Before{__shfl_sync(FULL_MASK, w.blk, k), __shfl_sync(FULL_MASK, w.row, k), t + k};
    }
    t = stop < 32 ? t + stop : min(t + 32, t_end);
    return w;
}

// How a window's rows lie in a warp.
template <int D, int B>
struct Rows {
    static constexpr int V = 8, LPR = D / V;    // elements per lane, lanes per row
    static constexpr int GPW = 32 / LPR;        // rows a warp at a time
    static constexpr int W = B * D > 16 * 128 ? (B * D) / (16 * 128) : 1;  // warps a page
    static constexpr int IT = B / (GPW * W);    // rows a lane
    static_assert(IT * 8 <= 64, "numbers a lane");
};

// The first n of a lane's IT rows of a head's keys or values (n uniform; the others zero): by times f are
// their numbers.  in(i, a, b) gives row i's chunks, angles its place in the rows of the table.
template <typename T, int D, int B, bool INTERLEAVED, bool ONE, typename In>
__device__ __forceinline__ void make_rows(bool is_k, const In& in, const float* angles, int R, bool norm,
                                          const uint64_t (&wa)[2], const uint64_t (&wb)[2], const LanePart& at, float eps,
                                          uint64_t (&f)[Rows<D, B>::IT][4], float (&by)[Rows<D, B>::IT]) {
    constexpr int IT = Rows<D, B>::IT, N = ONE ? 1 : IT, STEP = Rows<D, B>::GPW * D;
    uint2 a, b;
    if (!is_k) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint64_t x[2], y[2];
            in(i, a, b);
            Chunk8<T>::unpack(a, x);
            Chunk8<T>::unpack(b, y);
            f[i][0] = x[0];
            f[i][1] = x[1];
            f[i][2] = y[0];
            f[i][3] = y[1];
            by[i] = 1.f;
        }
    } else if (R == D) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            in(i, a, b);
            make_key<T, D, INTERLEAVED, Turning::ALL>(a, b, angles + i * STEP, R, norm, wa, wb, at, eps, f[i], by[i]);
        }
    } else if (R > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            in(i, a, b);
            make_key<T, D, INTERLEAVED, Turning::SOME>(a, b, angles + i * STEP, R, norm, wa, wb, at, eps, f[i], by[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            in(i, a, b);
            make_key<T, D, INTERLEAVED, Turning::NONE>(a, b, angles + i * STEP, R, norm, wa, wb, at, eps, f[i], by[i]);
        }
    }
#pragma unroll
    for (int i = N; i < IT; ++i) {
        by[i] = 0.f;
        f[i][0] = f[i][1] = f[i][2] = f[i][3] = 0;
    }
}

// The largest of m and the sizes of a lane's eight numbers of a row (a NaN is left out).
__device__ __forceinline__ float largest(const uint64_t (&f)[4], float m = 0.f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        unpack2(f[k], a, b);
        asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(a), "f"(b));
    }
    return m;
}

// A lane's eight numbers of a row, times x, into its places of the row.
__device__ __forceinline__ void store_row(uint8_t* out, int lo_at, int hi_at, const uint64_t (&f)[4], float x,
                                          bool real) {
    const uint64_t x2 = pack2(x, x);
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2(mul2(f[k], x2), v[2 * k], v[2 * k + 1]);
    const uint32_t lo = e4m3x4_of_floats(v[0], v[1], v[2], v[3]), hi = e4m3x4_of_floats(v[4], v[5], v[6], v[7]);
    if (real) {
        *reinterpret_cast<uint32_t*>(out + lo_at) = lo;
        *reinterpret_cast<uint32_t*>(out + hi_at) = hi;
    }
}

// The scales of a window's pages and their values, from the rows' numbers by[i] f[i] of one head.  `had`:
// lane j's page's scale before, where row j begins a run; tops and hads: this page's, in shared memory,
// which two warps of a page share behind barrier `bar`; staged: room for the warp's rows of values, from
// where a bulk copy brings a run of neighbouring rows to its page (none: stored directly).
template <int D, int B>
__device__ __forceinline__ void store_window(const Window& w, uint64_t (&f)[Rows<D, B>::IT][4],
                                             float (&by)[Rows<D, B>::IT], int part, const LanePart& at, bool real,
                                             uint8_t* pool, float* scales, unsigned page, uint32_t had, float* tops,
                                             uint32_t* hads, int bar, unsigned int* err,
                                             unsigned char* staged = nullptr) {
    using L = Rows<D, B>;
    constexpr int IT = L::IT, GPW = L::GPW, W = L::W, LPR = L::LPR;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = at.l;
    auto none = [&](int i) { return ((w.run >> ((part * IT + i) * GPW)) & ((1u << GPW) - 1)) == 0; };
    auto mine = [&](int i) { return ((w.run >> ((part * IT + i) * GPW + sub)) & 1) != 0; };
    const bool single = __popc(w.leaders & w.run) == 1;  // one run: nothing differs from row to row
    const bool in_run = (w.run >> lane) & 1, leads = in_run && w.lead == lane;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const float m = by[i] * largest(f[i]);
        if (mine(i)) most = fmaxf(most, m);
    }
    if (__any_sync(FULL_MASK, most > FLT_MAX)) {  // infinities are left out too, and become NaN
        most = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float a, b;
                unpack2(f[i][k], a, b);
                if (!(fabsf(a) * by[i] <= FLT_MAX)) a = __int_as_float(0x7fffffff);
                if (!(fabsf(b) * by[i] <= FLT_MAX)) b = __int_as_float(0x7fffffff);
                f[i][k] = pack2(a, b);
            }
            if (mine(i)) most = fmaxf(most, by[i] * largest(f[i]));
        }
    }
    float top = most;
    if (single) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        if (W > 1 && lane == 0) tops[part] = top;
    } else {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (none(i)) continue;
            float m = fmaxf(by[i] * largest(f[i]), 0.f);
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
            if (l == 0) tops[(part * IT + i) * GPW + sub] = m;
        }
    }
    if constexpr (W > 1) {
        if (part == 0) hads[lane] = had;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(32 * W) : "memory");
        had = hads[lane];
    } else {
        __syncwarp();
    }
    if (single) {
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (W > 1) top = fmaxf(top, tops[k]);
    } else {
        top = in_run ? tops[lane] : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(FULL_MASK, top, o);
            if (lane - o >= w.lead) top = fmaxf(top, x);
        }
        top = __shfl_sync(FULL_MASK, top, w.last);
    }
    had = __shfl_sync(FULL_MASK, had, w.lead);
    const bool ok = real && in_run && had != Q8_LOCKED;
    if (real && leads && !ok) set_error(err, PKV_DEVERR_SLOT);
    const float old = __uint_as_float(had), need = q8_scale_for(top);
    const float s = w.lead_row > 0 ? fmaxf(old, need) : need;  // (a scale that is NaN counts as none)
    // (of a power of two exactly, and without a division: but for 2^127, whose reciprocal has no place among the
    // normal numbers)
    const int bits = __float_as_int(s);
    const bool simple = (bits & 0x7fffff) == 0 && bits != 0x7f000000;
    const float inv = simple ? __int_as_float(0x7f000000 - bits) : 1.f / s;
    unsigned grown = __ballot_sync(FULL_MASK, ok && leads && w.lead_row > 0 && s > old);
    for (; grown != 0; grown &= grown - 1) {
        const int j = __ffs(grown) - 1, row0 = __shfl_sync(FULL_MASK, w.row, j);
        const unsigned rows_j = __ballot_sync(FULL_MASK, in_run && w.lead == j);
        const float ratio = __shfl_sync(FULL_MASK, old / s, j);
        uint8_t* const codes = pool + (size_t)__shfl_sync(FULL_MASK, page, j) * (B * D);
        for (int r = part * GPW + sub; r < B; r += W * GPW) {
            const int k = j + r - row0;
            if (k < j || k > 31 || !((rows_j >> k) & 1))
                round_again(reinterpret_cast<uint2*>(codes + r * D) + l, ratio);
        }
    }
    const unsigned stored = __ballot_sync(FULL_MASK, ok);
    if (single) {  // rows behind one another in one page
        const int j = __ffs(w.run & w.leaders) - 1, r0 = part * IT * GPW;
        const float x = __shfl_sync(FULL_MASK, inv, j);
        uint8_t* const out = pool + (size_t)__shfl_sync(FULL_MASK, page, j) * (B * D) +
                             (__shfl_sync(FULL_MASK, w.row, j) - j + r0) * D;
        if (staged != nullptr && stored == w.run && j == 0 && (w.run & (w.run + 1)) == 0) {
            if (lane == 0) bulk_wait_read<0>();  // the copy before has read its rows
            __syncwarp();
            const bool swap = sub & 1;  // (so that the rows of a warp meet in no bank)
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const uint64_t x2 = pack2(x * by[i], x * by[i]);
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) unpack2(mul2(f[i][k], x2), v[2 * k], v[2 * k + 1]);
                const uint32_t lo = e4m3x4_of_floats(v[0], v[1], v[2], v[3]);
                const uint32_t hi = e4m3x4_of_floats(v[4], v[5], v[6], v[7]);
                unsigned char* const row = staged + (i * GPW + sub) * D;
                *reinterpret_cast<uint32_t*>(row + (swap ? at.hi : at.lo)) = swap ? hi : lo;
                *reinterpret_cast<uint32_t*>(row + (swap ? at.lo : at.hi)) = swap ? lo : hi;
            }
            fence_proxy_async_shared();
            __syncwarp();
            const int rows = min(__popc(w.run) - r0, IT * GPW);
            if (lane == 0) {
                if (rows > 0) bulk_s2g(out, smem_addr(staged), rows * D);
                bulk_commit();
            }
        } else {
#pragma unroll
            for (int i = 0; i < IT; ++i)
                store_row(out + (i * GPW + sub) * D, at.lo, at.hi, f[i], x * by[i],
                          (stored >> ((part * IT + i) * GPW + sub)) & 1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r0 = (part * IT + i) * GPW, r = r0 + sub;
            if (((stored >> r0) & ((1u << GPW) - 1)) == 0) continue;
            const float x = __shfl_sync(FULL_MASK, inv, r) * by[i];
            uint8_t* const out =
                pool + (size_t)__shfl_sync(FULL_MASK, page, r) * (B * D) + __shfl_sync(FULL_MASK, w.row, r) * D;
            store_row(out, at.lo, at.hi, f[i], x, (stored >> r) & 1);
        }
    }
    if (ok && leads && part == 0) atomicExch(reinterpret_cast<unsigned int*>(scales + page), __float_as_uint(s));
}

template <typename T, bool INTERLEAVED>
__device__ __forceinline__ LanePart lane_part(int l, int R) {
    LanePart at;
    at.l = l;
    at.turns = l * 8 < R;
    at.lo = INTERLEAVED || !at.turns ? l * 8 : l * 4;
    at.hi = INTERLEAVED || !at.turns ? at.lo + 4 : at.lo + R / 2;
    return at;
}

template <typename T>
__device__ __forceinline__ void load_weights(const void* w, const LanePart& at, uint64_t (&wa)[2], uint64_t (&wb)[2]) {
    wa[0] = wa[1] = wb[0] = wb[1] = pack2(1.f, 1.f);
    if (w == nullptr) return;
    Chunk8<T>::unpack(__ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + at.lo)), wa);
    Chunk8<T>::unpack(__ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + at.hi)), wb);
}

}  // namespace

// (Runs one after another in a CTA took 44 us for 512 decoding requests, windows of many runs 13.)
// Few tokens, whose time is one row's way through the kernel: the first q_ctas CTAs have the q rows of a
// token each; of the others, every `heads` have the runs that begin in `rows` rows, and a warp one page's
// rows, all in flight.  The warps share the window's rows of the rotation table in shared memory.
template <typename T, int D, int B, bool INTERLEAVED>
__global__ void __launch_bounds__(Q8_KV_WARPS * 32, Q8_CTAS_PER_SM)
q8_write_kernel(const RopeParams p, float* k_scale, float* v_scale, int q_ctas, int heads, int rows) {
    using L = Rows<D, B>;
    constexpr int IT = L::IT, GPW = L::GPW, W = L::W;
    __shared__ __align__(16) float angles[B * D];
    __shared__ float tops[Q8_KV_WARPS / W][32];
    __shared__ uint32_t hads[Q8_KV_WARPS / W][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L::LPR;
    const int Hkv = p.num_kv_heads, R = p.rotary_dim;
    const LanePart at = lane_part<T, INTERLEAVED>(lane % L::LPR, R);
    if ((int)blockIdx.x < q_ctas) {
        turn_queries<T, D, INTERLEAVED>(p, at, blockIdx.x);
        return;
    }
    const int cta = (int)blockIdx.x - q_ctas, part = warp % W, unit = warp / W;
    const int first_u = cta % heads * (Q8_KV_WARPS / W), u = first_u + unit;
    const bool real = u < 2 * Hkv, is_k = u < Hkv;
    const int head = real ? (is_k ? u : u - Hkv) : 0;
    float* const scales = is_k ? k_scale : v_scale;
    uint8_t* const pool = static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool);
    const long long stride = is_k ? p.k_stride : p.v_stride;
    uint64_t wa[2], wb[2];
    load_weights<T>(p.k_weight, at, wa, wb);
    const int t_begin = cta / heads * rows, t_end = min(t_begin + rows, p.num_tokens);
    Before before = before_row<B>(p, t_begin);
    for (int t = t_begin; t < t_end;) {
        const int t_now = t;
        const Window w = find_window<B>(p, load_row(p, t + lane), before, t, t_end, threadIdx.x == 0);
        if (w.run == 0) continue;
        // the scale of each run's page, and no other run at that page from here on
        const unsigned page = (unsigned)max(w.blk, 0) * Hkv + head;  // (pages are 1 KB or more)
        uint32_t had = 0;
        if (real && part == 0 && (w.run & w.leaders) >> lane & 1)
            had = atomicExch(reinterpret_cast<unsigned int*>(scales + page), Q8_LOCKED);
        // this lane's chunks of rows (part * IT + i) * GPW + sub
        uint2 a[IT], b[IT];
        const T* const base =
            static_cast<const T*>(is_k ? p.k : p.v) + (t_now + part * IT * GPW + sub) * stride + head * D;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            a[i] = b[i] = make_uint2(0u, 0u);
            if ((w.run >> ((part * IT + i) * GPW + sub)) & 1) {
                a[i] = __ldcs(reinterpret_cast<const uint2*>(base + i * GPW * stride + at.lo));
                b[i] = __ldcs(reinterpret_cast<const uint2*>(base + i * GPW * stride + at.hi));
            }
        }
        if (R > 0 && first_u < Hkv) {
            for (int r = warp; r < B; r += Q8_KV_WARPS) {
                const int pr = __shfl_sync(FULL_MASK, w.pos, r);
                if ((w.run >> r) & 1)
                    for (int i = lane * 4; i < R; i += 128)
                        *reinterpret_cast<float4*>(angles + r * D + i) =
                            __ldg(reinterpret_cast<const float4*>(p.cos_sin + (size_t)pr * R + i));
            }
        }
        __syncthreads();
        const bool several = (w.run >> GPW) != 0;
        uint64_t f[IT][4];
        float by[IT];
        // (rows that are not of a run are made from anything, and not used)
        const float* const turn = angles + (part * IT * GPW + sub) * D;
        auto in = [&](int i, uint2& x, uint2& y) {
            x = a[i];
            y = b[i];
        };
        if (several)
            make_rows<T, D, B, INTERLEAVED, false>(is_k, in, turn, R, p.k_weight != nullptr, wa, wb, at, p.eps, f, by);
        else
            make_rows<T, D, B, INTERLEAVED, true>(is_k, in, turn, R, p.k_weight != nullptr, wa, wb, at, p.eps, f, by);
        store_window<D, B>(w, f, by, part, at, real, pool, scales, page, had, tops[unit], hads[unit], 1 + unit, p.err);
        __syncthreads();  // before the next window's rows of the table and maxima
    }
}

// Many tokens: CTAs that stay, with the keys and values of up to 8 heads, a page a warp (or two), window by
// window.  A window's rows come by one tensor copy each for k and v, a window ahead like its rows of the
// table and the pages' scales, and a run's values go out by one copy a page.  All this is with the warps
// of values, which take less work than keys; the last one also finds the windows, two ahead, from slots
// that it loads before its own window.
constexpr int Q8_STREAM_WARPS = 16, Q8_FOUND = 4;

template <int D, int B>
struct StreamSmem {
    static constexpr int OUT = B * D / Rows<D, B>::W;  // a warp's values of a window
    // two stages of k and v rows of `heads` heads and of table rows, and the values
    __host__ __device__ static constexpr int rows(int heads) { return B * heads * D * 2; }
    __host__ __device__ static constexpr int stage(int heads) { return 2 * rows(heads) + B * D * 4; }
    __host__ __device__ static constexpr int bytes(int heads) {
        return 2 * stage(heads) + 2 * heads * Rows<D, B>::W * OUT;
    }
};

template <typename T, int D, int B, bool INTERLEAVED>
__global__ void __launch_bounds__(Q8_STREAM_WARPS * 32, 1)
q8_stream_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                 const RopeParams p, float* k_scale, float* v_scale, int heads, int slices, int rows) {
    using L = Rows<D, B>;
    using S = StreamSmem<D, B>;
    constexpr int IT = L::IT, GPW = L::GPW, W = L::W;
    extern __shared__ __align__(128) unsigned char stream_smem[];
    struct Found {
        int t;
        unsigned run, leaders;
        int blk[32], row[32], pos[32], lead[32], last[32], lead_row[32];
    };
    __shared__ Found found[Q8_FOUND];
    __shared__ float tops[Q8_STREAM_WARPS / W][32];
    __shared__ uint32_t hads[Q8_STREAM_WARPS / W][32];
    __shared__ __align__(8) uint64_t bars[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L::LPR, warps = 2 * heads * W;
    const int Hkv = p.num_kv_heads, R = p.rotary_dim;
    const int t_begin = (int)blockIdx.x / slices * rows, t_end = min(t_begin + rows, p.num_tokens);
    const int head0 = (int)blockIdx.x % slices * heads, n_heads = min(heads, Hkv - head0);
    const uint32_t bar0 = smem_addr(bars);
    if (threadIdx.x == 0) {
        mbar_init(bar0, 1);
        mbar_init(bar0 + 8, 1);
        mbar_init_fence();
    }
    const LanePart at = lane_part<T, INTERLEAVED>(lane % L::LPR, R);
    const int part = warp % W, unit = warp / W;
    const bool is_k = unit < heads;
    const int h = is_k ? unit : unit - heads;   // of this slice
    const bool real = h < n_heads;
    float* const scales = is_k ? k_scale : v_scale;
    uint8_t* const pool = static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool);
    uint64_t wa[2], wb[2];
    load_weights<T>(p.k_weight, at, wa, wb);
    unsigned char* const out = stream_smem + 2 * S::stage(heads) + warp * S::OUT;
    const uint64_t policy = l2_evict_first_policy();  // the projections are not read again

    int t = t_begin;
    RawRow raw = load_row(p, t + lane);
    Before before = before_row<B>(p, t);
    auto find = [&](int i) {
        Found& x = found[i % Q8_FOUND];
        Window w;
        w.run = 0;
        int t_now = t;
        while (t < t_end && w.run == 0) {
            t_now = t;
            w = find_window<B>(p, raw, before, t, t_end, lane == 0);
            if (w.run == 0) raw = load_row(p, t + lane);
        }
        if (w.run != 0) {
            x.blk[lane] = w.blk; x.row[lane] = w.row; x.pos[lane] = w.pos;
            x.lead[lane] = w.lead; x.last[lane] = w.last; x.lead_row[lane] = w.lead_row;
        }
        if (lane == 0) {
            x.t = t_now;
            x.run = w.run;
            x.leaders = w.leaders;
        }
        __syncwarp();
    };
    auto bring = [&](int i) {  // this warp's share of window i's rows
        const Found& x = found[i % Q8_FOUND];
        const unsigned run = x.run;
        if (is_k || run == 0) return;
        const uint32_t bar = bar0 + 8 * (i & 1), stage = smem_addr(stream_smem + (i & 1) * S::stage(heads));
        if (warp == heads * W && umma::elect_one()) {
            mbar_arrive_expect_tx(bar, 2 * S::rows(heads));
            tma_load_3d(stage, &tmap_k, 0, head0, x.t, bar, policy);
            tma_load_3d(stage + S::rows(heads), &tmap_v, 0, head0, x.t, bar, policy);
        }
        for (int r = warp - heads * W; r < B; r += heads * W)
            if (((run >> r) & 1) && 4 * lane < R)
                cp_async16(stage + 2 * S::rows(heads) + (r * D + 4 * lane) * 4,
                           p.cos_sin + (size_t)x.pos[r] * R + 4 * lane);
    };
    // the scale of each run's page, and no other run at that page from here on
    auto lock = [&](int i) -> uint32_t {
        const Found& x = found[i % Q8_FOUND];
        if (!real || part != 0 || !((x.run & x.leaders) >> lane & 1)) return 0u;
        float* const at = scales + ((unsigned)x.blk[lane] * Hkv + head0 + h);
        return atomicExch(reinterpret_cast<unsigned int*>(at), Q8_LOCKED);
    };
    const bool finds = warp == warps - 1;
    if (finds) find(0);
    __syncthreads();
    bring(0);
    __syncwarp();
    uint32_t had = lock(0);
    if (finds) {
        raw = load_row(p, t + lane);
        find(1);
    }
    cp_async_wait_all();
    __syncthreads();
    for (int i = 0; found[i % Q8_FOUND].run != 0; ++i) {
        const Found& x = found[i % Q8_FOUND];
        bring(i + 1);
        __syncwarp();
        if (finds) raw = load_row(p, t + lane);
        Window w;
        w.run = x.run; w.leaders = x.leaders;
        w.blk = x.blk[lane]; w.row = x.row[lane]; w.lead_row = x.lead_row[lane];
        w.lead = x.lead[lane]; w.last = x.last[lane];
        const unsigned page = (unsigned)max(w.blk, 0) * Hkv + head0 + (real ? h : 0);
        if (!mbar_wait_short(bar0 + 8 * (i & 1), (i >> 1) & 1)) set_error(p.err, PKV_DEVERR_TIMEOUT);
        __syncwarp();
        // (rows that are not of a run are made from anything, and not used)
        const unsigned char* const stage = stream_smem + (i & 1) * S::stage(heads);
        const T* const row = reinterpret_cast<const T*>(stage + (is_k ? 0 : S::rows(heads))) +
                             ((part * IT * GPW + sub) * heads + h) * D;
        auto in = [&](int k, uint2& a, uint2& b) {
            a = *reinterpret_cast<const uint2*>(row + k * GPW * heads * D + at.lo);
            b = *reinterpret_cast<const uint2*>(row + k * GPW * heads * D + at.hi);
        };
        uint64_t f[IT][4];
        float by[IT];
        make_rows<T, D, B, INTERLEAVED, false>(
            is_k, in, reinterpret_cast<const float*>(stage + 2 * S::rows(heads)) + (part * IT * GPW + sub) * D, R,
            p.k_weight != nullptr, wa, wb, at, p.eps, f, by);
        store_window<D, B>(w, f, by, part, at, real, pool, scales, page, had, tops[unit], hads[unit], 1 + unit, p.err,
                           out);
        had = lock(i + 1);  // (not before: the fence in there would wait for it)
        if (finds) find(i + 2);
        cp_async_wait_all();  // this warp's rows of the next window's table
        __syncthreads();
    }
    if (lane == 0) bulk_wait_read<0>();  // the CTA must not end with copies still reading its shared memory
    // q's kernel, beside which this one may run and of which it needs nothing, is done when this one is
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

namespace {

// k or v seen as [tokens][heads][D]: a box is `heads` heads of `rows` tokens, as they lie.
template <typename T>
bool encode_rows_map(CUtensorMap* map, const void* base, long long stride, const RopeParams& p, int heads, int rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.num_kv_heads, (cuuint64_t)p.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)p.head_dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {(cuuint32_t)p.head_dim, (cuuint32_t)heads, (cuuint32_t)rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, Mma<T>::TMA_TYPE, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int B, bool INTERLEAVED>
cudaError_t launch_q8_write_tdbi(const RopeParams& p, float* k_scale, float* v_scale, cudaStream_t stream) {
    constexpr int W = Rows<D, B>::W, UNITS = Q8_KV_WARPS / W;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (p.num_tokens < Q8_MANY_TOKENS) {
        const long long heads = (2ll * p.num_kv_heads + UNITS - 1) / UNITS;
        const long long few = (p.num_tokens + Q8_FEW_ROWS - 1) / Q8_FEW_ROWS * heads;
        const int rows = few <= (long long)Q8_CTAS_PER_SM * sms ? Q8_FEW_ROWS : Q8_GROUP_ROWS;
        const long long ctas = p.num_tokens + ((long long)p.num_tokens + rows - 1) / rows * heads;
        if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
        q8_write_kernel<T, D, B, INTERLEAVED>
            <<<(unsigned)ctas, Q8_KV_WARPS * 32, 0, stream>>>(p, k_scale, v_scale, p.num_tokens, (int)heads, rows);
        return cudaGetLastError();
    }
    // a CTA per SM (two of few warps), each with a stretch of the rows and an even share of the heads
    constexpr int MOST = Q8_STREAM_WARPS / (2 * W);
    const int slices = (p.num_kv_heads + MOST - 1) / MOST, heads = (p.num_kv_heads + slices - 1) / slices;
    const int warps = 2 * heads * W;
    auto kernel = q8_stream_kernel<T, D, B, INTERLEAVED>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamSmem<D, B>::bytes(MOST));
    if (e != cudaSuccess) return e;
    const long long want = (long long)sms * (warps <= Q8_STREAM_WARPS / 2 ? 2 : 1);
    long long rows = ((long long)p.num_tokens * slices + want - 1) / want;
    rows = (rows + B - 1) / B * B;
    const long long ctas = (p.num_tokens + rows - 1) / rows * slices;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    CUtensorMap tk, tv;
    if (!encode_rows_map<T>(&tk, p.k, p.k_stride, p, heads, B) ||
        !encode_rows_map<T>(&tv, p.v, p.v_stride, p, heads, B))
        return cudaErrorNotSupported;
    RopeParams q = p;  // the q rows alone
    q.num_kv_heads = 0;
    e = launch_rope_write(q, std::is_same<T, __half>::value ? PKV_F16 : PKV_BF16, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = StreamSmem<D, B>::bytes(heads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tk, tv, p, k_scale, v_scale, heads, slices, (int)rows);
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
