// chunk.cuh -- causal attention of ragged chunks of new tokens over the paged cache, on the
// fifth-generation tensor cores ("Serving models with vLLM", section "How it works:
// continuous batching": chunked prefill; each request brings its own number of new tokens).
//
// For query j of request s (n_s queries, context c_s counting them), head h:
//   out = softmax(scale q . K_s[0..lim)^T) V_s[0..lim),   lim = c_s - n_s + 1 + j,
// zero when lim <= 0; a NaN or infinite score makes its row NaN.  The G heads of a kv head share
// its K and V, so the rows of one kv head are (query, head) pairs and a CTA takes two tiles of 128
// of them (row r of a tile is query r / G, head r % G) against the pages in steps of 128 tokens:
// every staged K and V tile serves 256 rows.  One pass, running maximum and sum per row.
//
// A small kernel first lists the pieces of work (chunk_plan.cu): tile pair x kv head, cut
// along the context where there would be too few of them; the CTAs of this kernel, one per
// SM, take pieces from that list in order until it is empty.  Sixteen warps, fixed roles:
//   0-3, 4-7  softmax of tile 0 and of tile 1
//   8         takes the next piece; tensor copies of K and V pages into a ring of stages
//   9         one lane issues the MMAs, for the two tiles in turn:
//               S_t = Q_t . K_j^T            128 x 128 in tensor memory
//               O_t += P_t . V_j             P_t written over S_t by the softmax
//             so that one tile's softmax runs while the tensor cores work for the other.
//             Before a piece's last P.V the warp zeroes the V rows of the last 16-token copy
//             past the last position the piece may see (they may hold anything; their
//             weights are zero, and 0 * NaN is not)
//   10        tensor copies of the query tiles
//   11        none (fills the warpgroup)
//   12-15     output of a finished piece, while the others are at the next one
// A piece takes one of three forms by its rows:
//   more than 128  both tiles;
//   17 to 128      one tile: the even and the odd steps' scores take the two tiles' places, so
//                  a step's scores are ready when the softmax of the step before ends;
//   up to 16       (decoding requests) each of warps 0-3 has all rows and a quarter of the
//                  tokens of every step, and the four results are joined at the end.
// The reference of a row follows its maximum, and is raised only when a step's maximum exceeds
// the one it was set by by more than 8 in base 2, so O is rescaled rarely; every term of a row uses
// the same reference.  P enters its product rounded to the pool's type (at most half a step,
// 2^-8 of the value in bf16 and 2^-11 in fp16, like the output's own rounding); with a 32-bit
// output it enters as a rounded part and the rounded remainder, in two products.  fp16 has full
// steps from 2^-14 on and half a step of 2^-25 below, so there the reference lies 7 below the
// maximum: weights go up to 2^15, those from 2^-21 of the largest on keep their 11 bits, and no
// weight is off by more than 2^-32 of the largest.  Scores, maxima, sums and O are held in 32 bits.
// The tensor cores cut a sum's low bits off, always towards zero, so a row's O in tensor memory
// falls behind its sum by up to 2^-23 a product of 16 tokens (weights alike over 2^20 tokens: by
// 1 %).  So after every CHUNK_SUM_STEPS steps of a piece O and the sum are added to 32-bit totals in
// the workspace and begin at zero again: off by 8 * 256 * 2^-23 = 2^-12 at most, whatever the
// length (2^-11 with a 32-bit output, whose weights take two products; measured there, weights and
// values alike over 2^20 tokens: 2^-12.7).  A row's sum is one of sums of steps.
//
// What bounds it, measured.  Two full tiles: a step has 2048 cycles of MMAs and takes about
// 2650, the way of one tile once round: its softmax (1500 cycles: scores from tensor memory 310,
// 128 exponentials 920), the second half of P.V (256), Q.K^T (512) and three hand-overs.  8192
// tokens from the first on, 32 / 8 heads of 128, bf16: 360 us, 1.53 PFLOP/s (0.80 of cuBLAS);
// 500 tokens over 130,500: 712 to 745 us at the power cap, about 1.47 PFLOP/s.  What got it there,
// each for that prompt:
//   MMAs and copies issued under elect.sync and not under lane == 0 (67 cycles an MMA, 100 a
//     copy there): 470 -> 411 us, and with V's copies three-dimensional (one for both halves of
//     16 tokens; K's halves have to lie apart) 394;
//   one thread issuing both tiles' MMAs and not one each, which run interleaved, so that both
//     tiles' exponentials compete for the same units at the same time: 394 -> 373;
//   registers so that the softmax does not spill: 373 -> 364; output by warps of its own: 352.
// (One setmaxnreg for warps 8 to 11 and sums of steps brought it to 360.)  With a 32-bit output, whose
// P.V is twice as long, the prompt takes 624 us.
// Few rows over long contexts: 64 KB of K and V a step bound it, 1960 cycles where the HBM's share of
// an SM is 2790 (32 requests over 60,000 tokens, 64 / 8 heads: 1135 us, 6.9 TB/s).  Over short ones
// a piece's fixed cycles do, because copies run at most two pieces ahead of the output: 200 requests of
// one query over 300 tokens, 32 / 8 heads 61.5 us, 1.7 times their bytes; 16 over 1500 24 us, 1.7.
// Tried and slower: 16 softmax warps that share rows and exchange maxima; exponentials begun
// with the old reference before the maximum is known; merging cut items in this kernel; the first
// scores of the next piece issued before the last products of this one (48 requests, 70 % decoding,
// 40 / 40 heads: 268 us, 256 without), and its record and first block fetched early (260).
// Over a pool held in 8 bits (Q8) the pages come in as e4m3 values, and warps 12-15 turn each tile into the
// 16-bit numbers of the products between its copy and them, ahead of the MMAs by as many stages as there
// are, and the next piece's first tiles before they put out this one's results.  Keys become the queries'
// type, values fp16: an e4m3 value times a power of two is exact in either.  fp16 has no room for any
// page's scale, so keys enter relative to the largest scale of their step, which goes into the factor of the
// scores, and values relative to a power of two, the base, by which O is held until its output.  The base
// moves only where fp16 would not hold a step's values by it, and O is scaled with it, in 32 bits; so the
// weights are the same whatever the scales are.  What bounds it: shared memory, which the products read at
// 128 bytes a cycle while scores are made (1540 of a step's cycles), the copies, reads and stores of the
// conversion take 1020 more of, and the conversion's issue slots beside the softmax's.  (Both figures from
// the bytes.)  Besides, the code of all roles together passes what an SM keeps of it: code that is never run
// cost up to 10 % by where it put the rest (500 tokens over 130,500, with 64 more instructions there 960 us).
// The prompt takes 465 us (359 from 16 bits), 863,000 cycles an SM for 219 steps, pieces' beginnings and ends
// among them; 500 tokens over 130,500 855 us (689 to 703); fp16 455 and 850 us.
// Every wait is bounded; a CTA that gives up sets PKV_DEVERR_TIMEOUT and returns its tensor
// memory.
#pragma once

#include <climits>
#include <type_traits>

#include "decode_mma.cuh"
#include "q8.cuh"
#include "umma.cuh"

namespace pkv {

constexpr int CHUNK_THREADS = 512;
// Registers per thread: 128 at launch; the softmax warps take what the others give back
// (256 * 184 + 128 * 72 + 128 * 72 = 512 * 128).
constexpr int CHUNK_REGS_SOFTMAX = 184, CHUNK_REGS_OTHERS = 72, CHUNK_REGS_OUTPUT = 72;
// The maximum of a row, in base 2, that a step's weights are judged by, how far below it the
// reference is set, and how far it may exceed the reference.  The largest weight of fp16 has to stay
// below 2^16: its maximum is rounded up, so that the one product and sum of a weight's exponent,
// which leaves out the maximum's rounding, cannot exceed what was judged.
template <typename T>
struct ChunkReference {
    static constexpr float BELOW = 0.f, RAISE = 8.f;
    __device__ __forceinline__ static float scaled(float x, float scale_log2) { return x * scale_log2; }
};
template <>
struct ChunkReference<__half> {
    static constexpr float BELOW = 7.f, RAISE = 15.f;
    __device__ __forceinline__ static float scaled(float x, float scale_log2) { return __fmul_ru(x, scale_log2); }
};
// Rows up to which a piece's steps are spread over four warps: 200 requests with 1-5 queries, 32 / 8
// heads, contexts about 300: 79 us (93 with 4 rows).
constexpr int CHUNK_FEW_ROWS = 16;

// Q8: pages arrive as e4m3 values, and the stages hold them as numbers of the products' types.
// Steps whose references (below) are kept: a step's are written when its copies are issued, at most
// RAW_STAGES + STAGES stages before its products, and read by the softmax, at most two steps later.
constexpr int Q8_STEP_RING = 16;
// Bases of values, as powers of two: what a piece begins with (pages whose largest number lies between 2^-14 and
// 448 * 2^-1 need no other), and the least one, also relative to the largest so far: O is scaled up by no more.
constexpr int Q8_FIRST_BASE = -8, Q8_LEAST_BASE = -60;
constexpr int Q8_PART_POWER = 40;
template <int D, bool Q8>
struct ChunkSmem {
    static constexpr int BOXES = D / 64;                  // 128-byte columns of a row
    static constexpr int BOX = 128 * 128;                 // one of a 128-row tile
    static constexpr int TILE = BOXES * BOX;              // a tile of Q, K or V
    // Q8, D = 128: a tile's e4m3 rows land where the second half of its numbers will be, and become
    // numbers there, row by row.  (With a ring of their own and three stages of numbers, a step's keys had
    // no room until the values before the last were done with: a prompt took 489 us and not 465.)
    // D = 64: rows of half a line, in a ring of their own.
    static constexpr bool IN_PLACE = Q8 && D == 128;
    static constexpr int STAGES = D == 128 ? 5 : Q8 ? 6 : 8;
    static constexpr int RAW_STAGES = Q8 ? (IN_PLACE ? STAGES : 8) : 0;  // of e4m3 values, as their barriers count
    static constexpr int RAW_TILE = 128 * D;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = 2 * TILE;
    static constexpr int RAW_OFF = KV_OFF + STAGES * TILE;
    static constexpr int SCALE_OFF = RAW_OFF + (IN_PLACE ? 0 : RAW_STAGES * RAW_TILE);  // float [RAW_STAGES][8 copies]
    static constexpr int STEP_OFF = SCALE_OFF + RAW_STAGES * 32;       // float4 [Q8_STEP_RING]
    static constexpr int BAR_OFF = STEP_OFF + (Q8 ? Q8_STEP_RING * 16 : 0);
    static constexpr int NBARS = 2 * STAGES + 31 + 2 * RAW_STAGES;
    static constexpr int PIECE_OFF = BAR_OFF + ((NBARS * 8 + 15) / 16) * 16;
    static constexpr int STAT_OFF = PIECE_OFF + 2 * 32;  // float [2 tiles][m, l][128 rows]
    static constexpr int BASE_OFF = STAT_OFF + 2 * 2 * 128 * 4;  // Q8: int [4], the bases that pieces end with
    static constexpr int TMEM_SLOT_OFF = BASE_OFF + 16;
    static constexpr int BYTES = TMEM_SLOT_OFF + 16;
    // tensor memory columns: S_0, S_1 (P over them), O_0, O_1; of a piece with few rows P has the
    // last 128 columns
    static constexpr uint32_t FEW_P_COL = 384;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t O_COL = 256;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(4 * CHUNK_FEW_ROWS * D * 4 <= TILE, "the warps' rows meet in the second Q tile");
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// x, as a value made here: addresses derived from it are made where they are used.  Kept in
// registers across the loops, those of all the products took the MMA warp 192 bytes past its
// registers, and an 8192-token prompt 402 us and not 357.
__device__ __forceinline__ uint32_t made_here(uint32_t x) {
    asm volatile("" : "+r"(x));
    return x;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float v;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
    return v;
}

// 2 to a whole number from -126 to 127.
__device__ __forceinline__ float two_to(int x) { return __int_as_float((x + 127) << 23); }

// Adds the row's total, kept at `kept` (its 16-byte columns 128 apart; O's, then the sum and their
// reference), to its O at o_t and its sum l.  TO_TOTAL: the sums become the total (the `first` ones are O and
// l alone), and O zero.  Q8: the total is held by a base of 2^40, O by base[0]'s.  Returns the sum.  Out of
// line: inlined, it cost steps that never come here (8192-token prompt 365 us, 360 so).
template <int D, bool TO_TOTAL, bool Q8>
__device__ __noinline__ float add_total(uint32_t o_t, float4* kept, float m_ref, float l, const int* base,
                                        bool first) {
    const uint32_t zeros[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    float2* const sum_and_ref = reinterpret_cast<float2*>(kept + D / 4 * 128);
    const float2 before = first ? make_float2(0.f, m_ref) : *sum_and_ref;
    float f = before.y == m_ref ? 1.f : fast_exp2(before.y - m_ref);
    l = fmaf(before.x, f, l);
    if (TO_TOTAL) *sum_and_ref = make_float2(l, m_ref);
    const float unit = Q8 && TO_TOTAL ? two_to(*base - Q8_PART_POWER) : 1.f;
    if (Q8 && !TO_TOTAL) f *= two_to(Q8_PART_POWER - *base);
#pragma unroll 1
    for (int d = 0; d < D; d += 16) {
        float4 v[4];
        float o[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = first ? make_float4(0.f, 0.f, 0.f, 0.f) : kept[(d / 4 + k) * 128];
        umma::ld16(o_t + d, o);
        if (Q8 && TO_TOTAL) {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= unit;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[4 * k] = fmaf(v[k].x, f, o[4 * k]);
            o[4 * k + 1] = fmaf(v[k].y, f, o[4 * k + 1]);
            o[4 * k + 2] = fmaf(v[k].z, f, o[4 * k + 2]);
            o[4 * k + 3] = fmaf(v[k].w, f, o[4 * k + 3]);
        }
        if (TO_TOTAL) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                kept[(d / 4 + k) * 128] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            umma::st16(o_t + d, zeros);
        } else {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k]);
            umma::st16(o_t + d, w);
        }
    }
    umma::wait_st();
    umma::fence_before_sync();
    return l;
}

// The base of a step's values, from their pages' scales (a lane each; 0: none), the base of the steps before
// and the largest one so far.  Whole warps.  Out of line: seldom called.
static __device__ __noinline__ int moved_base(int scale, int base, int base_top) {
    const int most = __reduce_max_sync(FULL_MASK, scale);
    const int least = __reduce_min_sync(FULL_MASK, scale == 0 ? INT_MAX : (scale & 0x7fffff) == 0 ? scale : 0);
    const int power = (most >> 23) - 127 + ((most & 0x7fffff) != 0);  // of two, that reaches the largest
    if (power <= base + 7 && base <= max((least >> 23) - 127 + 15, power)) return base;
    return min(max(power - 4, max(base_top, 0) + Q8_LEAST_BASE), 126);
}

// One step of a row: its 128 scores from tensor memory at s_t, the running reference m_ref and
// the sum (in two parts), its O at o_t scaled where the reference rose (once phase_o of
// bar_o says that the products before are done; 0: known), and its weights written over the
// scores, the halves handed on at bar_lo and bar_hi.
// Q8: moved is what O is multiplied with besides, where the base of the values moves with this step.
// edge: the warp has scores that their rows do not see.
template <typename T, int D, bool SPLIT_P, bool Q8, typename Edge>
__device__ __forceinline__ bool softmax_step(uint32_t s_t, uint32_t o_t, int seen, const Edge edge, bool has_o,
                                             float scale_log2, float moved, float& m_ref, uint64_t& sum2,
                                             uint32_t bar_lo, uint32_t bar_hi, uint32_t bar_o,
                                             uint32_t phase_o) {
    constexpr int N = CHUNK_TILE, HALF = N / 2;
    const int lane = threadIdx.x & 31;
    uint32_t raw[N];
    float top[8];  // eight chains of three-input maxima
    umma::ld32_async(s_t, raw);
    umma::ld32_async(s_t + 32, raw + 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        umma::wait_ld(raw + h * HALF);
        umma::wait_ld(raw + h * HALF + 32);
        if (h == 0) {  // the second half arrives while the first is looked at
            umma::ld32_async(s_t + HALF, raw + HALF);
            umma::ld32_async(s_t + HALF + 32, raw + HALF + 32);
        }
        if (edge) {
#pragma unroll
            for (int k = h * HALF; k < (h + 1) * HALF; ++k)
                if (k >= seen) raw[k] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int k0 = h * HALF + c;
            if (h == 0) top[c] = __uint_as_float(raw[k0]);
#pragma unroll
            for (int k = h == 0 ? k0 + 8 : k0; k + 8 < (h + 1) * HALF; k += 16)
                top[c] = max3(top[c], __uint_as_float(raw[k]), __uint_as_float(raw[k + 8]));
            if (h == 0) top[c] = fmaxf(top[c], __uint_as_float(raw[HALF - 8 + c]));
        }
    }
    using Ref = ChunkReference<T>;
    const float most = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7]));
    const float cm = Ref::scaled(most, scale_log2);
    const bool need = cm - m_ref > Ref::RAISE;
    float alpha = 1.f;
    if (need) {
        alpha = fast_exp2(m_ref - (cm - Ref::BELOW));
        m_ref = cm - Ref::BELOW;
    }
    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
    const uint64_t scale2 = pack2(scale_log2, scale_log2), neg2 = pack2(neg, neg);
    sum2 = mul2(sum2, pack2(alpha, alpha));
    uint64_t step2[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < N; c += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(raw[c + k]), __uint_as_float(raw[c + k + 1])), scale2, neg2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            step2[(k >> 1) & 1] = add2(step2[(k >> 1) & 1], pack2(a, b));
            hi[k / 2] = Mma<T>::pack(a, b);
            if (SPLIT_P) lo[k / 2] = Mma<T>::pack(a - Mma<T>::round_trip(a), b - Mma<T>::round_trip(b));
        }
        umma::st16(s_t + c / 2, hi);
        if (SPLIT_P) umma::st16(s_t + HALF + c / 2, lo);
        if (c == HALF - 32) {
            // rows whose reference rose, or all where the base moves: scale their O, complete through the
            // step before
            if (has_o && (__any_sync(FULL_MASK, need) || (Q8 && moved != 1.f))) {
                if (Q8) alpha *= moved;
                if (bar_o != 0) {
                    if (!__all_sync(FULL_MASK, mbar_wait_short(bar_o, phase_o & 1))) return false;
                    umma::fence_after_sync();
                }
#pragma unroll
                for (int d = 0; d < D; d += 16) {
                    float o[16];
                    umma::ld16(o_t + d, o);
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * alpha);
                    umma::st16(o_t + d, w);
                }
            }
            umma::wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_lo);
        }
    }
    sum2 = add2(sum2, add2(step2[0], step2[1]));
    umma::wait_st();
    umma::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_hi);
    return true;
}

// One step of a row of a piece with few rows: this warp's 32 scores at s_t, the reference, sum
// and O as in softmax_step, the weights to p_t.  The caller hands them on.
template <typename T, int D, bool Q8>
__device__ __forceinline__ bool few_rows_step(uint32_t s_t, uint32_t p_t, uint32_t o_t, int seen, bool has_o,
                                              float scale_log2, float moved, float& m_ref, float& l, uint32_t bar_o,
                                              uint32_t phase_o) {
    uint32_t raw[32];
    umma::ld32_async(s_t, raw);
    umma::wait_ld(raw);
    if (__any_sync(FULL_MASK, seen < 32)) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (k >= seen) raw[k] = 0xff800000u;  // -inf
    }
    float top[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        top[c] = fmaxf(__uint_as_float(raw[c]), __uint_as_float(raw[c + 28]));
#pragma unroll
        for (int k = c + 4; k < 28; k += 8)
            top[c] = max3(top[c], __uint_as_float(raw[k]), __uint_as_float(raw[k + 4 < 28 ? k + 4 : k]));
    }
    using Ref = ChunkReference<T>;
    const float most = max3(top[0], top[1], fmaxf(top[2], top[3]));
    const float cm = Ref::scaled(most, scale_log2);
    const bool need = cm - m_ref > Ref::RAISE;
    if (__any_sync(FULL_MASK, need) || (Q8 && moved != 1.f)) {
        float alpha = 1.f;
        if (need) {
            alpha = fast_exp2(m_ref - (cm - Ref::BELOW));
            m_ref = cm - Ref::BELOW;
        }
        l *= alpha;
        if (Q8) alpha *= moved;
        if (has_o) {  // rows whose reference rose (all, where the base moves): O is complete through the step before
            if (!__all_sync(FULL_MASK, mbar_wait_short(bar_o, phase_o & 1))) return false;
            umma::fence_after_sync();
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                float o[16];
                umma::ld16(o_t + d, o);
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * alpha);
                umma::st16(o_t + d, w);
            }
        }
    }
    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
    const uint64_t scale2 = pack2(scale_log2, scale_log2), neg2 = pack2(neg, neg);
    uint64_t sum2[2] = {0, 0};
    uint32_t hi[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        float a, b;
        unpack2(fma2(pack2(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), scale2, neg2), a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        sum2[(k >> 1) & 1] = add2(sum2[(k >> 1) & 1], pack2(a, b));
        hi[k / 2] = Mma<T>::pack(a, b);
    }
    umma::st16(p_t, hi);
    float part[4];
    unpack2(sum2[0], part[0], part[1]);
    unpack2(sum2[1], part[2], part[3]);
    const float sum = (part[0] + part[1]) + (part[2] + part[3]);
    l += sum;
    umma::wait_st();
    umma::fence_before_sync();
    __syncwarp();
    return true;
}

// A raw tile (128 tokens of D e4m3 values, rows behind one another) into a stage's K or V tile of 16-bit
// numbers, times a factor per copy of 16 tokens, by four warps: 16 values a lane at a time, which become
// two 16-byte columns.  Eight lanes read 128 bytes in a row, and write eight different columns of the
// 128-byte swizzle (with D = 128 the lanes of the second half store their odd column first).  To fp16,
// factors that it holds, as those between powers of two are, multiply in fp16; others, and all to bf16, in
// 32 bits, so that each number is rounded once.
enum class Factor { HALF, SINGLE };

template <typename M, int D, Factor BY, int UNROLL, bool IN_PLACE>
__device__ __forceinline__ void numbers_by(const unsigned char* raw, const float* factor, unsigned char* tile,
                                           bool is_v, int w, int lane) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;    // lanes a row, rows a warp at a time
    constexpr int STEPS = 128 / (4 * ROWS);
    const int m = lane % LANES, box = m / 4, col = 2 * (m % 4);
    const bool swap = box == 1;
    // rows (i * 4 + w) * ROWS + lane / LANES: whole copies of 16 rows a step apart
    const int row0 = w * ROWS + lane / LANES, r = row0 % CHUNK_TOKENS, b0 = row0 / CHUNK_TOKENS;
    constexpr int COPIES = 4 * ROWS / CHUNK_TOKENS;     // copies a step
    const int copy = is_v ? CHUNK_TOKENS * D * 2 : CHUNK_TOKENS * 128;
    unsigned char* at = tile + b0 * copy + box * (is_v ? CHUNK_TOKENS * 128 : 128 * 128) + r * 128;
    const int stride = COPIES * copy;
    at += ((col + swap) ^ (r & 7)) << 4;
    const int other = ((((col + swap) ^ 1) ^ (r & 7)) << 4) - (((col + swap) ^ (r & 7)) << 4);
    // (in place: the row's place in the second half of the numbers)
    raw = IN_PLACE ? tile + b0 * copy + (is_v ? CHUNK_TOKENS * 128 : 128 * 128) + r * 128 + m * 16
                   : raw + row0 * D + m * 16;
    const int raw_stride = IN_PLACE ? stride : 4 * ROWS * D;
    // (short loops: the code of all roles shares the instruction cache; whole, they cost a prompt 10 %)
#pragma unroll 1
    for (int i = 0; i < STEPS; i += UNROLL) {
        uint4 x[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) x[u] = *reinterpret_cast<const uint4*>(raw + (i + u) * raw_stride);
        if (IN_PLACE) __syncwarp();  // a row is read by the lanes that write over it, before they do
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t out[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) f16x4_of_e4m3x4(in[k], out[2 * k], out[2 * k + 1]);
            const float s = factor[b0 + (i + u) * COPIES];
            const __half2 h2 = __half2half2(__float2half_rn(s));
            const uint64_t s2 = pack2(s, s);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (BY == Factor::HALF) {
                    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&out[k]), h2);
                    out[k] = *reinterpret_cast<const uint32_t*>(&v);
                } else {
                    const float2 v = float2_of_f16x2(out[k]);
                    float a, c;
                    unpack2(mul2(pack2(v.x, v.y), s2), a, c);
                    out[k] = Mma<M>::pack(a, c);
                }
            }
            const uint4 lo4 = make_uint4(out[0], out[1], out[2], out[3]);
            const uint4 hi4 = make_uint4(out[4], out[5], out[6], out[7]);
            *reinterpret_cast<uint4*>(at + (i + u) * stride) = swap ? hi4 : lo4;
            *reinterpret_cast<uint4*>(at + (i + u) * stride + other) = swap ? lo4 : hi4;
        }
    }
}

template <typename M, int D, bool IN_PLACE>
__device__ __forceinline__ void numbers_of_tile(const unsigned char* raw, const float* factor, unsigned char* tile,
                                                bool is_v, int w, int lane) {
    const float mine = factor[lane % 8];
    if (!std::is_same<M, __half>::value)
        numbers_by<M, D, Factor::SINGLE, 2, IN_PLACE>(raw, factor, tile, is_v, w, lane);
    else if (__all_sync(FULL_MASK, __half2float(__float2half_rn(mine)) == mine))
        numbers_by<__half, D, Factor::HALF, 2, IN_PLACE>(raw, factor, tile, is_v, w, lane);
    else
        numbers_by<__half, D, Factor::SINGLE, 1, IN_PLACE>(raw, factor, tile, is_v, w, lane);
}

template <typename T, int D, bool SPLIT_P, bool Q8>
__global__ void __launch_bounds__(CHUNK_THREADS, 1)
chunk_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_q32,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const ChunkParams p) {
    using L = ChunkSmem<D, Q8>;
    constexpr int NS = L::STAGES, KS = D / 16;
    constexpr int KV_WARP = 8, MMA_WARP = 9, Q_WARP = 10, OUT_WARP = 12;
    constexpr int CONSUMERS = 8 + 2 + 4;  // arrivals that free a slot of the piece ring
    // The type of the weights and values: over 8-bit pools fp16, which holds every e4m3 value and takes
    // fewest instructions to reach.  Keys have the queries' type.
    using M = typename std::conditional<Q8, __half, T>::type;
    constexpr bool KEYS_F16 = std::is_same<T, __half>::value;
    constexpr uint32_t FMT = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t FMT_O = std::is_same<M, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t IDESC_S = umma::idesc_f16(FMT, false, 128, CHUNK_TILE);
    const uint32_t idesc_s = IDESC_S | (p.negate ? umma::IDESC_NEGATE_A : 0u);
    constexpr uint32_t IDESC_O = umma::idesc_f16(FMT_O, true, 128, D);

    // the swizzle repeats every 1024 bytes; no static shared memory lies before this array
    extern __shared__ __align__(1024) unsigned char chunk_smem[];
    unsigned char* smem = chunk_smem;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t q_s = sbase + L::Q_OFF, ring = sbase + L::KV_OFF, bar0 = sbase + L::BAR_OFF;
    const int G = p.group, QPT = 128 / G;  // heads per kv head, queries per tile
    // barriers: K / V stage landed and free; Q tile landed and free; a piece's last P.V
    // done; piece published and read; every MMA done; the P.V of an even or odd step
    // of a piece with one tile of queries done (a barrier each: a warp may be a step ahead of
    // another one, with two products still to come, and one barrier's parity would not tell
    // them apart)
    auto kv_full = [&](int st) { return bar0 + 8 * st; };
    auto kv_empty = [&](int st) { return bar0 + 8 * (NS + st); };
    constexpr int NB = 2 * NS;
    auto q_full = [&](int t) { return bar0 + 8 * (NB + t); };
    auto q_empty = [&](int t) { return bar0 + 8 * (NB + 2 + t); };
    auto pv_done = [&](int t) { return bar0 + 8 * (NB + 6 + t); };
    auto piece_full = [&](int i) { return bar0 + 8 * (NB + 8 + i); };
    auto piece_empty = [&](int i) { return bar0 + 8 * (NB + 10 + i); };
    const uint32_t all_done = bar0 + 8 * (NB + 12);
    auto pv_step = [&](int b) { return bar0 + 8 * (NB + 4 + b); };
    // S tile ready and half of a P tile written: i < 2 of tile i, i = 2, 3 of the even and odd
    // steps of a piece with one tile of queries (barriers of their own, because the second
    // tile's warps take no part in them)
    auto s_full = [&](int i) { return bar0 + 8 * (NB + 13 + i); };
    auto p_full = [&](int i, int h) { return bar0 + 8 * (NB + 17 + 2 * i + h); };
    // a tile's m and l are in shared memory; its O (and m and l) have been read; the four warps'
    // rows of a piece with few rows are in shared memory, and have been read
    auto stat_full = [&](int t) { return bar0 + 8 * (NB + 25 + t); };
    auto o_free = [&](int t) { return bar0 + 8 * (NB + 27 + t); };
    const uint32_t few_done = bar0 + 8 * (NB + 29), few_read = bar0 + 8 * (NB + 30);
    // Q8: a tile of e4m3 values landed, and read
    constexpr int NR = L::RAW_STAGES;
    auto raw_full = [&](int st) { return bar0 + 8 * (NB + 31 + st); };
    auto raw_empty = [&](int st) { return bar0 + 8 * (NB + 31 + NR + st); };
    float* raw_scale = reinterpret_cast<float*>(smem + L::SCALE_OFF);
    // of the n-th step of this CTA: what its keys are smaller by (fp16 ones), what O is multiplied with where the
    // base of its values is another than that of the step before (1 otherwise), and that base
    float4* step_ref = reinterpret_cast<float4*>(smem + L::STEP_OFF);
    float* stats = reinterpret_cast<float*>(smem + L::STAT_OFF);  // + 256 t: m, + 128: l
    // Q8: the base that the n-th piece of this CTA ends with (whoever takes a piece is done with the one before the
    // last, and pieces are published two ahead: four places)
    int* piece_base = reinterpret_cast<int*>(smem + L::BASE_OFF);
    auto is_few = [&](const ChunkPiece& x) {
        return !SPLIT_P && x.queries * G <= CHUNK_FEW_ROWS && x.kt1 > x.kt0;
    };
    ChunkPiece* pieces = reinterpret_cast<ChunkPiece*>(smem + L::PIECE_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::TMEM_SLOT_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int st = 0; st < NS; ++st) {
            mbar_init(kv_full(st), Q8 ? 4 : 1);
            mbar_init(kv_empty(st), 1);
        }
        for (int st = 0; st < NR; ++st) {
            mbar_init(raw_full(st), 1);
            mbar_init(raw_empty(st), 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full(t), 1);
            mbar_init(q_empty(t), 1);
            for (int i = t; i < 4; i += 2) {
                mbar_init(s_full(i), 1);
                mbar_init(p_full(i, 0), 4);
                mbar_init(p_full(i, 1), 4);
            }
            mbar_init(pv_done(t), 1);
            mbar_init(pv_step(t), 1);
            mbar_init(stat_full(t), 4);
            mbar_init(o_free(t), 4);
            mbar_init(piece_full(t), 1);
            mbar_init(piece_empty(t), CONSUMERS);
        }
        mbar_init(all_done, 1);
        mbar_init(few_done, 4);
        mbar_init(few_read, 4);
        mbar_init_fence();
    }
    if (warp == MMA_WARP) umma::alloc(smem_addr(tmem_slot), L::TMEM_COLS);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // the list of pieces is written by the kernel before this one in the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // The i-th piece of this CTA, published by the copy warp; false when there is none left
    // (or the wait ran out).
    bool ok = true;
    auto next_piece = [&](int i, ChunkPiece& pc) -> bool {
        ok = __all_sync(FULL_MASK, mbar_wait_short(piece_full(i & 1), (i >> 1) & 1));
        if (!ok) return false;
        pc = pieces[i & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_empty(i & 1));
        return pc.kv_head >= 0;
    };

    // Each warpgroup sets its registers once, all four warps at the same place (setmaxnreg is
    // undefined where a warpgroup's warps do not take it alike), and inside its own branch: where
    // branches meet again, the compiler would hold both to the smaller number.
    if (warp >= KV_WARP && warp < OUT_WARP) {
        regs_dec<CHUNK_REGS_OTHERS>();
        if (warp == KV_WARP) {
            // ---- pieces, and the pages of each: K then V of every 128-token step
            const uint64_t policy = l2_evict_normal_policy();
            const ChunkPiece first_piece = p.pieces[blockIdx.x];  // the list has a place for each CTA
            const int n_pieces = p.header[0];
            const int B = p.block_size, Hkv = p.num_kv_heads;
            const int far_row = p.num_blocks * Hkv * B;  // past the pools: copies bring zeros
            constexpr int NBOX = CHUNK_TILE / CHUNK_TOKENS;  // 16-token copies of a step; lane b finds b's block
            uint32_t it = 0;  // stages filled so far
            int idx = blockIdx.x;
            for (int i = 0;; ++i) {
                ChunkPiece pc;
                pc.kv_head = -1;
                if (idx < n_pieces) pc = i == 0 ? first_piece : p.pieces[idx];
                if (i >= 2) {
                    ok = __all_sync(FULL_MASK, mbar_wait_short(piece_empty(i & 1), ((i >> 1) - 1) & 1));
                    if (!ok) break;
                }
                if (lane == 0) {
                    pieces[i & 1] = pc;
                    mbar_arrive(piece_full(i & 1));  // release: the record is visible to its waiters
                }
                if (pc.kv_head < 0) break;
                int next = 0;
                if (lane == 0) next = atomicAdd(p.header + 2, 1);
                const int32_t* bt_row = p.block_tables + (size_t)pc.seq * p.max_blocks_per_seq;
                const int tok_end = pc.lim0 + pc.queries - 1;
                auto row_of = [&](int kt) -> int {  // pool row of this lane's copy in step kt
                    const int t = kt * CHUNK_TILE + lane * CHUNK_TOKENS;
                    if (kt >= pc.kt1 || t >= tok_end || lane >= NBOX) return far_row;
                    const int phys = __ldg(bt_row + t / B);
                    if ((unsigned)phys >= (unsigned)p.num_blocks) {
                        set_error(p.err, PKV_DEVERR_BLOCK_ID);
                        return far_row;
                    }
                    return (phys * Hkv + pc.kv_head) * B + t % B;
                };
                int row = row_of(pc.kt0);
                // Q8: the scales of this lane's copy (far_row: a multiple of B, past the last page)
                float scale_now[2] = {0.f, 0.f}, scale_next[2] = {0.f, 0.f};
                auto scales_of = [&](int row, float (&s)[2]) {
                    s[0] = s[1] = 0.f;
                    if (row != far_row) {
                        s[0] = __ldg(p.k_scale + row / B);
                        s[1] = __ldg(p.v_scale + row / B);
                    }
                };
                int row_then = 0;
                if constexpr (Q8) {
                    scales_of(row, scale_now);
                    row_then = row_of(pc.kt0 + 1);
                }
                // In fp16 a step's keys enter the products relative to the largest scale among their pages, which
                // goes into the scores' factor: numbers of pages far smaller than that lose bits in fp16's last
                // steps, 2^-33 of the step's largest.  Values enter relative to 2^base, and O is a sum of such.
                // The base stays while fp16 holds the step's values by it: up to 2^7 times the base in scale, and
                // down to 2^-15 of it where scales are powers of two (e4m3's steps of 2^-9 times that are 2^-24),
                // otherwise no less than it; pages smaller than 2^-15 of the step's largest do not count.  So it
                // moves seldom, and then to 2^-4 of the largest.
                float factor[2] = {0.f, 0.f};
                int base = Q8_FIRST_BASE, base_top = Q8_FIRST_BASE;
                auto make_factors = [&] {
                    // (sizes as whole numbers, which are ordered alike; lanes without a page have zeros)
                    const int own = __float_as_int(fabsf(scale_now[1])), before = base;
                    const bool fits = (own & 0x7fffff) == 0 && (unsigned)own - ((base - 15 + 127) << 23) <= 22u << 23;
                    if (!__all_sync(FULL_MASK, fits || own == 0)) {
                        base = moved_base(own, base, base_top);
                        base_top = max(base_top, base);
                    }
                    const float moved = two_to(max(before - base, -126));
                    float keys = 0.f;
                    if (KEYS_F16)
                        keys = __int_as_float(__reduce_max_sync(FULL_MASK, __float_as_int(fabsf(scale_now[0]))));
                    factor[0] = !KEYS_F16 ? scale_now[0] : keys > 0.f ? scale_now[0] / keys : 0.f;
                    factor[1] = scale_now[1] * two_to(-base);
                    if (lane == 0) {
                        step_ref[(it / 2) % Q8_STEP_RING] = make_float4(keys, moved, __int_as_float(base), 0.f);
                        piece_base[i & 3] = base;
                    }
                };
                for (int kt = pc.kt0; kt < pc.kt1 && ok; ++kt) {
                    const int row_next = row_of(Q8 ? kt + 2 : kt + 1);
                    if constexpr (Q8) scales_of(row_then, scale_next);
                    int rows[NBOX];
#pragma unroll
                    for (int b = 0; b < NBOX; ++b) rows[b] = __shfl_sync(FULL_MASK, row, b);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        if constexpr (Q8) {
                            const int st = it % NR;
                            if (it >= NR) {
                                ok = __all_sync(FULL_MASK, mbar_wait_short(L::IN_PLACE ? kv_empty(st) : raw_empty(st),
                                                                           ((it / NR) - 1) & 1));
                                if (!ok) break;
                            }
                            // the copies first, while the scales are on their way, and the arrival that tells of
                            // both when these are there
                            if (umma::elect_one()) {
                                const uint32_t full = raw_full(st);
                                uint32_t dst = sbase + L::RAW_OFF + st * L::RAW_TILE, copy = CHUNK_TOKENS * D;
                                if (L::IN_PLACE) {  // into the second half of each row's numbers
                                    dst = ring + st * L::TILE + (kv == 0 ? L::BOX : CHUNK_TOKENS * 128);
                                    copy = kv == 0 ? CHUNK_TOKENS * 128 : CHUNK_TOKENS * D * 2;
                                }
#pragma unroll
                                for (int b = 0; b < NBOX; ++b)
                                    tma_load_2d(dst + b * copy, kv == 0 ? &tmap_k : &tmap_v, 0, rows[b], full, policy);
                            }
                            __syncwarp();
                            if (kv == 0) make_factors();
                            if (lane < NBOX) raw_scale[st * NBOX + lane] = factor[kv];
                            __syncwarp();
                            if (umma::elect_one()) mbar_arrive_expect_tx(raw_full(st), L::RAW_TILE);
                            __syncwarp();
                            continue;
                        }
                        const int st = it % NS;
                        if (it >= NS) {
                            ok = __all_sync(FULL_MASK, mbar_wait_short(kv_empty(st), ((it / NS) - 1) & 1));
                            if (!ok) break;
                        }
                        // from one elected thread: copies issued by 16 lanes at once took about
                        // 100 cycles each, and the whole kernel the time of its copies
                        if (umma::elect_one()) {
                            const uint32_t full = kv_full(st), dst = ring + st * L::TILE;
                            mbar_arrive_expect_tx(full, L::TILE);
#pragma unroll
                            for (int b = 0; b < NBOX; ++b) {
                                if (kv == 0) {
                                    // K tile: 128-byte columns of 128 rows
#pragma unroll
                                    for (int x = 0; x < L::BOXES; ++x)
                                        tma_load_2d(dst + x * L::BOX + b * CHUNK_TOKENS * 128, &tmap_k, x * 64,
                                                    rows[b], full, policy);
                                } else {
                                    // V tile: a copy's columns behind one another (one K step of P.V)
                                    tma_load_3d(dst + b * CHUNK_TOKENS * D * 2, &tmap_v, 0, rows[b], 0, full, policy);
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if constexpr (Q8) {
                        row = row_then;
                        row_then = row_next;
                        scale_now[0] = scale_next[0];
                        scale_now[1] = scale_next[1];
                    } else {
                        row = row_next;
                    }
                }
                if (!ok) break;
                idx = __shfl_sync(FULL_MASK, next, 0);
            }
            // the CTA must not end with copies still landing in its shared memory
            if constexpr (Q8) {
                for (uint32_t k = it > NR ? it - NR : 0; k < it; ++k) mbar_wait_short(raw_full(k % NR), (k / NR) & 1);
            } else {
                for (uint32_t k = it > NS ? it - NS : 0; k < it; ++k) mbar_wait_short(kv_full(k % NS), (k / NS) & 1);
            }
        } else if (warp == Q_WARP) {
            // ---- query tiles
            int loads[2] = {0, 0}, fews = 0;  // copies into each tile, pieces with few rows
            bool few_last = false;            // tile 1 was taken last by such a piece
            ChunkPiece pc;
            for (int i = 0; next_piece(i, pc); ++i) {
                if (pc.kt1 <= pc.kt0) continue;
                // a piece with few rows has them in tile 0 four times, 32 rows apart, and takes tile
                // 1 for the warps' results
                const bool few = is_few(pc);
                for (int t = 0; t < (few || pc.queries > QPT ? 2 : 1); ++t) {
                    if (t == 1 && few_last)
                        ok = __all_sync(FULL_MASK, mbar_wait_short(few_read, (fews - 1) & 1));
                    else if (loads[t] > 0)
                        ok = __all_sync(FULL_MASK, mbar_wait_short(q_empty(t), (loads[t] - 1) & 1));
                    if (!ok) break;
                    if (t == 1) few_last = few;
                    if (few && t == 1) {
                        ++fews;
                        continue;
                    }
                    ++loads[t];
                    if (umma::elect_one()) {
                        const uint32_t dst = q_s + t * L::TILE;
                        if (few) {
                            mbar_arrive_expect_tx(q_full(0), 4 * L::BOXES * (32 / G) * G * 128);
                            for (int w = 0; w < 4; ++w)
                                for (int x = 0; x < L::BOXES; ++x)
                                    tma_load_4d(dst + x * L::BOX + w * 32 * 128, &tmap_q32, 0, x, pc.kv_head * G,
                                                pc.token, q_full(0));
                        } else {
                            mbar_arrive_expect_tx(q_full(t), L::BOXES * QPT * G * 128);
                            for (int x = 0; x < L::BOXES; ++x)
                                tma_load_4d(dst + x * L::BOX, &tmap_q, 0, x, pc.kv_head * G, pc.token + t * QPT,
                                            q_full(t));
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            for (int t = 0; t < 2; ++t)
                if (loads[t] > 0) mbar_wait_short(q_full(t), (loads[t] - 1) & 1);
        } else if (warp == MMA_WARP) {
            // ---- MMA issue, the two tiles in turn: one thread for both, because MMAs issued by
            // two threads are interleaved, both tiles' scores are then complete at the same time
            // and their exponentials compete for the same units
            uint32_t total = 0;               // stages of the pieces so far
            int used[2] = {0, 0};             // Q tiles taken
            int steps[4] = {0, 0, 0, 0};      // P tiles taken, as s_full and p_full count them
            int outs[2] = {0, 0};             // pieces begun in O_0 and O_1
            // i: tile 0 or 1, or 2, 3 for an even or odd step of a piece with one tile of queries
            auto issue_s = [&](int i, int st) {  // S over the P just read: MMAs run in issue order
                const uint64_t k_desc = umma::sw128_desc(ring + st * L::TILE, 16, 1024);
                const uint64_t q_desc = umma::sw128_desc(made_here(q_s + (i == 1 ? L::TILE : 0)), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    const uint32_t off = ((kk >> 2) * L::BOX + (kk & 3) * 32) >> 4;  // start address field
                    umma::mma_f16(tmem + (i & 1) * CHUNK_TILE, q_desc + off, k_desc + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                umma::commit(s_full(i));  // also says that every P.V before is done
            };
            auto issue_pv = [&](int i, int st, bool first, bool few = false) -> bool {
                // V is N-major: 64-element columns 2048 apart, 8-token groups 1024, and a K step
                // is one copy's 16 tokens.  The first half's products run while the softmax still
                // works on the second half.
                const uint64_t v_desc = umma::sw128_desc(ring + st * L::TILE, CHUNK_TOKENS * 128, 1024);
                const uint32_t cols = made_here(tmem), o_t = cols + L::O_COL + (i == 1 ? D : 0);
                const uint32_t p_t =
                    cols + (few ? L::FEW_P_COL + (i & 1) * (CHUNK_TILE / 2) : (i & 1) * CHUNK_TILE);
                const uint32_t parity = steps[i]++ & 1;
                if (first) {  // the piece before has been read from O
                    int& o = outs[i == 1];
                    if (o > 0 && !mbar_wait_short(o_free(i == 1), (o - 1) & 1)) return false;
                    ++o;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!mbar_wait_short(p_full(i, h), parity)) return false;
                    umma::fence_after_sync();
#pragma unroll
                    for (int k = 4 * h; k < 4 * h + 4; ++k) {
                        const uint64_t bv = v_desc + (k * CHUNK_TOKENS * D * 2 >> 4);
                        umma::mma_f16_tmem_a(o_t, p_t + k * 8, bv, IDESC_O, (!first || k > 0) ? 1u : 0u);
                        if (SPLIT_P) umma::mma_f16_tmem_a(o_t, p_t + CHUNK_TILE / 2 + k * 8, bv, IDESC_O, 1u);
                    }
                }
                return true;
            };
            ChunkPiece pc;
            for (int i = 0; next_piece(i, pc); ++i) {
                const int n = pc.kt1 - pc.kt0;
                if (n <= 0) continue;
                const bool two = pc.queries > QPT, few = is_few(pc);
                int st = (int)(total % NS);  // next stage and its phase
                uint32_t phase = (total / NS) & 1;
                auto landed = [&] { return mbar_wait_short(kv_full(st), phase); };
                auto advance = [&] {
                    if (++st == NS) {
                        st = 0;
                        phase ^= 1;
                    }
                };
                if (!two) {
                    // one tile of queries: the scores of the even and the odd steps take the places
                    // of the two tiles', so that a step's scores are ready when the softmax of the
                    // step before ends
                    if (umma::elect_one()) {
                        auto stage = [&](int k) { return (int)((total + k) % NS); };
                        auto in = [&](int k) { return mbar_wait_short(kv_full(stage(k)), ((total + k) / NS) & 1); };
                        auto scores = [&](int j) -> bool {
                            if (!in(2 * j)) return false;
                            umma::fence_after_sync();
                            issue_s(2 + (j & 1), stage(2 * j));
                            if (j == n - 1) umma::commit(q_empty(0));
                            umma::commit(kv_empty(stage(2 * j)));
                            return true;
                        };
                        ok = mbar_wait_short(q_full(0), used[0] & 1) && scores(0) && (n == 1 || scores(1));
#pragma unroll 1
                        for (int j = 0; j < n - 1 && ok; ++j) {
                            ok = in(2 * j + 1) && issue_pv(2 + (j & 1), stage(2 * j + 1), j == 0, few);
                            if (!ok) break;
                            umma::commit(pv_step(j & 1));
                            umma::commit(kv_empty(stage(2 * j + 1)));
                            if (j + 2 < n) ok = scores(j + 2);
                        }
                    }
                } else if (umma::elect_one()) {
                    ok = landed();
                    if (ok) ok = mbar_wait_short(q_full(0), used[0] & 1);
                    if (ok) {
                        umma::fence_after_sync();
                        issue_s(0, st);
                        if (n == 1) umma::commit(q_empty(0));
                        ok = mbar_wait_short(q_full(1), used[1] & 1);
                        umma::fence_after_sync();
                        if (ok) issue_s(1, st);
                        if (n == 1) umma::commit(q_empty(1));
                        umma::commit(kv_empty(st));
                        advance();
                    }
#pragma unroll 1
                    for (int j = 0; j < n - 1 && ok; ++j) {
                        const int v_st = st;
                        ok = landed();
                        if (!ok) break;
                        advance();
                        ok = issue_pv(0, v_st, j == 0) && landed();
                        if (!ok) break;
                        umma::fence_after_sync();
                        issue_s(0, st);
                        if (j == n - 2) umma::commit(q_empty(0));
                        ok = issue_pv(1, v_st, j == 0);
                        if (!ok) break;
                        umma::commit(kv_empty(v_st));
                        issue_s(1, st);
                        if (j == n - 2) umma::commit(q_empty(1));
                        umma::commit(kv_empty(st));
                        advance();
                    }
                }
                ++used[0];
                used[1] += two;
                ok = __all_sync(FULL_MASK, ok);
                if (!ok) break;
                total += 2 * n;
                st = (int)((total - 1) % NS);  // every lane: the piece's last stage, V's
                phase = ((total - 1) / NS) & 1;
                if (chunk_has_tail(pc)) {
                    ok = __all_sync(FULL_MASK, landed());
                    if (!ok) break;
                    const int r0 = pc.lim0 + pc.queries - 1 - (pc.kt1 - 1) * CHUNK_TILE;
                    const int rows = CHUNK_TOKENS - r0 % CHUNK_TOKENS;
                    unsigned char* tile =
                        smem + L::KV_OFF + st * L::TILE + r0 / CHUNK_TOKENS * (CHUNK_TOKENS * D * 2);
                    for (int v = lane; v < rows * L::BOXES * 8; v += 32) {
                        const int r = r0 % CHUNK_TOKENS + v / (L::BOXES * 8), c = v % (L::BOXES * 8);
                        *reinterpret_cast<uint4*>(tile + (c / 8) * (CHUNK_TOKENS * 128) + r * 128 + (c % 8) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    umma::fence_smem_to_async();
                    __syncwarp();
                }
                if (!two) {
                    if (umma::elect_one()) {
                        ok = landed() && issue_pv(2 + ((n - 1) & 1), st, n == 1, few);
                        if (ok) umma::commit(pv_step((n - 1) & 1));
                        if (ok) umma::commit(kv_empty(st));
                    }
                } else if (umma::elect_one()) {
                    ok = landed() && issue_pv(0, st, n == 1);
                    if (ok) umma::commit(pv_done(0));
                    if (ok) {
                        ok = issue_pv(1, st, n == 1);
                        if (ok) umma::commit(pv_done(1));
                    }
                    if (ok) umma::commit(kv_empty(st));
                }
                ok = __all_sync(FULL_MASK, ok);
                if (!ok) break;
            }
            if (umma::elect_one()) {
                umma::commit(all_done);
                if (!mbar_wait_short(all_done, 0)) ok = false;
            }
            __syncwarp();
        }
    } else if (warp >= OUT_WARP) {
        regs_dec<CHUNK_REGS_OUTPUT>();
        // ---- output of both tiles, while the softmax warps are at the next piece: warp w of
        // these reads the rows that warps w and 4 + w worked on
        const int w = warp - OUT_WARP, r = w * 32 + lane;
        const uint32_t lane_tmem = tmem + ((uint32_t)(w * 32) << 16);
        const int hg = r % G;
        int even = 0, odd = 0;    // steps of pieces with one tile so far: the phases of pv_step
        int outs = 0, twos = 0;   // pieces so far, those with two tiles: of stat_full, pv_done
        int fews = 0;             // pieces with few rows: of few_done
        // Q8: these warps also make the stages' numbers, of a piece before its output and of the next
        // piece's first step too, so that its scores need not wait for that output.  (A stage that is
        // waited for here becomes free by products that no output is needed for.)
        uint32_t made = 0;  // stages so far
        auto make_stages = [&](int count) -> bool {
            for (int k = 0; k < count; ++k, ++made) {
                const int from = made % (NR > 0 ? NR : 1), st = made % NS;
                if (!__all_sync(FULL_MASK, mbar_wait_short(raw_full(from), (made / (NR > 0 ? NR : 1)) & 1)))
                    return false;
                if (!L::IN_PLACE && made >= NS &&
                    !__all_sync(FULL_MASK, mbar_wait_short(kv_empty(st), (made / NS - 1) & 1)))
                    return false;
                // (even ones are K's)
                const unsigned char* const raw = smem + L::RAW_OFF + from * L::RAW_TILE;
                unsigned char* const tile = smem + L::KV_OFF + st * L::TILE;
                if (KEYS_F16 || (made & 1))
                    numbers_of_tile<M, D, L::IN_PLACE>(raw, raw_scale + from * 8, tile, made & 1, w, lane);
                else
                    numbers_of_tile<T, D, L::IN_PLACE>(raw, raw_scale + from * 8, tile, false, w, lane);
                umma::fence_smem_to_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(kv_full(st));
                    if (!L::IN_PLACE) mbar_arrive(raw_empty(from));
                }
            }
            return true;
        };
        // Of the piece at work and the next one only their steps are needed here, so that the registers are
        // free for the numbers: the record stays where it is until the output.
        constexpr int AHEAD = NS - 1;
        int steps_next = 0;
        auto look_at = [&](int i) -> bool {
            ok = __all_sync(FULL_MASK, mbar_wait_short(piece_full(i & 1), (i >> 1) & 1));
            if (!ok) return false;
            const ChunkPiece& x = pieces[i & 1];
            steps_next = max(x.kt1 - x.kt0, 0);
            return x.kv_head >= 0;
        };
        ChunkPiece pc;
        bool any = Q8 && look_at(0);
        int ahead = 0;  // stages of the next piece that are made already
        for (int i = 0;; ++i) {
            if constexpr (Q8) {
                if (!any) break;
                ok = make_stages(2 * steps_next - ahead);
                if (!ok) break;
                any = look_at(i + 1);
                if (!ok) break;
                ahead = any ? min(AHEAD, 2 * steps_next) : 0;
                ok = make_stages(ahead);
                if (!ok) break;
                pc = pieces[i & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(piece_empty(i & 1));
            } else if (!next_piece(i, pc)) {
                break;
            }
            const int n = max(pc.kt1 - pc.kt0, 0);
            const bool two = pc.queries > QPT, direct = pc.part_row < 0, few = is_few(pc);
            if (!two) {
                even += (n + 1) / 2;
                odd += n / 2;
            }
            for (int t = 0; t < (two ? 2 : 1); ++t) {
                const uint32_t o_t = lane_tmem + L::O_COL + t * D;
                if (n > 0) {
                    // the sums first: then every product but the last of each barrier is done, and
                    // the parity tells
                    ok = __all_sync(FULL_MASK, mbar_wait_short(stat_full(t), (t == 0 ? outs : twos) & 1));
                    if (!ok) break;
                    const int last = (n - 1) & 1;
                    ok = __all_sync(FULL_MASK, two ? mbar_wait_short(pv_done(t), twos & 1)
                                                   : mbar_wait_short(pv_step(last), ((last ? odd : even) - 1) & 1));
                    if (!ok) break;
                    umma::fence_after_sync();
                }
                const float m = stats[256 * t + r];
                float l = n > 0 ? stats[256 * t + 128 + r] : 0.f;
                // Q8: O times its base; of a part of a row 2^-40 of that and of the sum, whose weights go up to
                // 2^15, so that values at the end of the range leave room for them
                float unit = 1.f, sum_unit = 1.f;
                if (Q8 && n > 0) {
                    sum_unit = direct ? 1.f : two_to(-Q8_PART_POWER);
                    unit = two_to(piece_base[i & 3]) * sum_unit;
                    l *= sum_unit;
                }
                if (few) {
                    // the four results of each row meet in the second Q tile; row r's 16-byte
                    // columns are turned by r, so that a warp's stores spread over the banks
                    const int rows = pc.queries * G;
                    constexpr int COLS = D / 4;
                    float4* rows_s = reinterpret_cast<float4*>(smem + L::Q_OFF + L::TILE);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        umma::ld16(o_t + c, o);
                        if (lane < rows) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                rows_s[(w * CHUNK_FEW_ROWS + lane) * COLS + (c / 4 + k + lane) % COLS] =
                                    make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        }
                        __syncwarp();
                    }
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(few_done);
                    ok = __all_sync(FULL_MASK, mbar_wait_short(few_done, fews & 1));
                    if (!ok) break;
                    for (int x = w; x < rows; x += 4) {
                        float M = -INFINITY, sum = 0.f, f[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) M = fmaxf(M, stats[y * 32 + x]);
                        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            f[y] = fast_exp2(stats[y * 32 + x] - ref);
                            sum = fmaf(f[y], stats[128 + y * 32 + x] * sum_unit, sum);
                        }
                        // zero for a row that sees nothing; a NaN or a sum of no weight is the result
                        const float inv = !direct ? 1.f : pc.lim0 + x / G > 0 ? 1.f / sum : 0.f;
                        const long long out_row =
                            ((long long)pc.token + x / G) * p.num_q_heads + pc.kv_head * G + x % G;
                        const long long part_row = (long long)pc.part_row + x;
                        if (lane < COLS) {
                            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float4 v = rows_s[(y * CHUNK_FEW_ROWS + x) * COLS + (lane + x) % COLS];
                                const float fw = f[y] * (inv * unit);
                                o.x = fmaf(fw, v.x, o.x);
                                o.y = fmaf(fw, v.y, o.y);
                                o.z = fmaf(fw, v.z, o.z);
                                o.w = fmaf(fw, v.w, o.w);
                            }
                            if (direct)
                                reinterpret_cast<uint2*>(static_cast<T*>(p.out) + out_row * D)[lane] =
                                    make_uint2(Mma<T>::pack(o.x, o.y), Mma<T>::pack(o.z, o.w));
                            else
                                reinterpret_cast<float4*>(p.part_o + part_row * D)[lane] = o;
                        }
                        if (!direct && lane == 0) {
                            p.part_m[part_row] = M;  // base 2
                            p.part_l[part_row] = sum;
                        }
                    }
                    // the second Q tile, O and the sums go back when all four have read them
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(few_read);
                        mbar_arrive(o_free(0));
                    }
                    ++fews;
                    break;
                }
                const int jq = t * QPT + r / G;  // query within the piece
                const bool valid = r < QPT * G && jq < pc.queries;
                if (__any_sync(FULL_MASK, valid)) {
                    const long long out_row = ((long long)pc.token + jq) * p.num_q_heads + pc.kv_head * G + hg;
                    const long long part_row = (long long)pc.part_row + (t * QPT * G + r);
                    // a row that sees nothing is zero, whatever O holds; a NaN in its sum, or no weight
                    // in it although it sees tokens (scores of -inf), is the result
                    const bool nothing = direct ? pc.lim0 + jq <= 0 : l == 0.f;
                    const float by = (direct ? 1.f / l : 1.f) * unit;
                    // once per piece: a loop that stays in the instruction cache
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        if (n > 0) umma::ld16(o_t + c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = nothing ? 0.f : o[k] * by;
                        if (!valid) {
                        } else if (direct && !SPLIT_P) {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + out_row * D + c);
#pragma unroll
                            for (int k = 0; k < 16; k += 8)
                                dst[k / 8] =
                                    make_uint4(Mma<T>::pack(o[k], o[k + 1]), Mma<T>::pack(o[k + 2], o[k + 3]),
                                               Mma<T>::pack(o[k + 4], o[k + 5]), Mma<T>::pack(o[k + 6], o[k + 7]));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(
                                direct ? static_cast<float*>(p.out) + out_row * D + c : p.part_o + part_row * D + c);
#pragma unroll
                            for (int k = 0; k < 16; k += 4)
                                dst[k / 4] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                        __syncwarp();
                    }
                    if (valid && !direct) {
                        p.part_m[part_row] = m;  // base 2
                        p.part_l[part_row] = l;
                    }
                }
                if (n > 0) {
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free(t));
                }
            }
            if (!ok) break;
            if (n > 0) {
                ++outs;
                twos += two;
            }
        }
    } else {
        regs_inc<CHUNK_REGS_SOFTMAX>();
        // ---- softmax of tile t: this thread's row is r
        const int t = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_t = lane_tmem + L::O_COL + t * D;
        const int jq = t * QPT + r / G;                // query within the piece
        int taken = 0, taken_even = 0, taken_odd = 0;  // S tiles so far: the phases of s_full and pv_step
        int outs = 0, twos = 0;  // pieces handed to the output warps, those with two tiles: of o_free
        uint32_t steps = 0;      // Q8: of the pieces before, as step_ref counts them
        // what the scores of step j of the piece are multiplied with (positive, though nothing be left of it:
        // hidden scores are -inf), what O is where the base of the values moves, and that base
        auto step_scale = [&](const float2& ref) -> float {
            if constexpr (!Q8 || !KEYS_F16) return p.scale_log2;
            return fmaxf(p.scale_log2 * ref.x, 1.2e-38f);
        };
        auto step_at = [&](int j) -> float2 {
            return Q8 ? *reinterpret_cast<const float2*>(step_ref + (steps + j) % Q8_STEP_RING) : make_float2(1.f, 1.f);
        };
        bool p_clear = false;    // the P columns of pieces with few rows hold zeros where they should
        // The row's totals of the steps before, in the workspace: O's, then the sum and their reference (not in
        // registers, which the steps need).
        auto kept = [&]() -> float4* {
            return reinterpret_cast<float4*>(p.totals) + (blockIdx.x * 2 + t) * (128 * (D / 4 + 1)) + r;
        };
        // before step j's softmax, its products so far done: O and the sum into the totals
        auto keep = [&](int j, float m_ref, float l) {
            const float4* const ref = step_ref + (steps + j - 1) % Q8_STEP_RING;
            add_total<D, true, Q8>(o_t, kept(), m_ref, l, Q8 ? reinterpret_cast<const int*>(ref) + 2 : nullptr,
                                   j == CHUNK_SUM_STEPS);
        };
        // at the end of piece i, all products done: the totals into O and the sum
        auto total = [&](int i, float m_ref, float l) -> float {
            return add_total<D, false, Q8>(o_t, kept(), m_ref, l, Q8 ? piece_base + (i & 3) : nullptr, false);
        };
        // waits for the products of the steps before step j (not yet taken), or of all of a piece
        auto products_before = [&](int j, bool two, bool all = false) -> bool {
            // (two tiles: the next scores are committed behind the products before them)
            const uint32_t bar = !two ? pv_step((j - 1) & 1) : all ? pv_done(t) : s_full(t);
            const int phase = !two ? ((j & 1) ? taken_even : taken_odd) - 1 : all ? twos : taken;
            if (!__all_sync(FULL_MASK, mbar_wait_short(bar, phase & 1))) return false;
            umma::fence_after_sync();
            return true;
        };
        // this row's m and l to the output warps
        auto hand_out = [&](float m, float l) -> bool {
            if (outs > 0) ok = __all_sync(FULL_MASK, mbar_wait_short(o_free(t), (outs - 1) & 1));
            if (!ok) return false;
            ++outs;
            stats[256 * t + r] = m;
            stats[256 * t + 128 + r] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(stat_full(t));
            return true;
        };
        ChunkPiece pc;
        for (int i = 0; next_piece(i, pc); ++i) {
            const int n = max(pc.kt1 - pc.kt0, 0);
            const bool two = pc.queries > QPT;
            if (n == 0 || (t == 1 && !two)) {  // one tile: the other warpgroup takes both S tiles
                steps += n;
                continue;
            }
            if (is_few(pc)) {
                // Few rows: warp w has them all, in its own 32 lanes, and of every step the tokens
                // 32 w .. 32 w + 31, its own reference, sum and O; its P holds zeros for the other
                // tokens.  A step's softmax takes a quarter of the time, and the step that of its
                // copies.
                const int rows = pc.queries * G, lim_w = pc.lim0 + min(lane, rows - 1) / G - warp * 32;
                const uint32_t p_t = lane_tmem + L::FEW_P_COL;
                if (!p_clear) {
                    // O_1 lies there: wait until it has been read.  (Tile 0 of the piece before
                    // first, so that at most one reading of O_1 is still to come and the parity
                    // tells which.)
                    if (outs > 0) ok = __all_sync(FULL_MASK, mbar_wait_short(o_free(0), (outs - 1) & 1));
                    if (ok && twos > 0) ok = __all_sync(FULL_MASK, mbar_wait_short(o_free(1), (twos - 1) & 1));
                    if (!ok) break;
                    umma::fence_after_sync();
                    const uint32_t zeros[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
                    for (int c = 0; c < CHUNK_TILE; c += 16) umma::st16(p_t + c, zeros);
                    umma::wait_st();
                    p_clear = true;
                }
                float m_ref = -INFINITY, l = 0.f;
                for (int j = 0; j < n && ok;) {
                    if (j > 0) {
                        ok = products_before(j, false);
                        if (!ok) break;
                        keep(j, m_ref, l);
                        l = 0.f;
                    }
                    for (const int end = min(n, j + CHUNK_SUM_STEPS); j < end; ++j) {
                        const int b = j & 1, phase = b ? taken_odd++ : taken_even++;
                        ok = __all_sync(FULL_MASK, mbar_wait_short(s_full(2 + b), phase & 1));
                        if (!ok) break;
                        umma::fence_after_sync();
                        const float2 ref = step_at(j);
                        const float by = step_scale(ref), moved = ref.y;
                        ok = few_rows_step<M, D, Q8>(lane_tmem + b * CHUNK_TILE + warp * 32,
                                                     p_t + b * (CHUNK_TILE / 2) + warp * 16, o_t,
                                                     lim_w - (pc.kt0 + j) * CHUNK_TILE, j > 0, by, moved, m_ref, l,
                                                     pv_step(b ^ 1), (b ? taken_even : taken_odd) - 1);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive(p_full(2 + b, 0));
                            mbar_arrive(p_full(2 + b, 1));
                        }
                    }
                }
                if (ok && n > CHUNK_SUM_STEPS) {
                    ok = products_before(n, false, true);
                    if (ok) l = total(i, m_ref, l);
                }
                steps += n;
                if (!ok || !hand_out(m_ref, l)) break;
                continue;
            }
            const bool busy = __any_sync(FULL_MASK, r < QPT * G && jq < pc.queries);
            const int lim = pc.lim0 + jq;
            float m_ref = -INFINITY;
            uint64_t sum2 = 0;  // the row's sum, in two parts
            auto sum = [&] {
                float a, b;
                unpack2(sum2, a, b);
                return a + b;
            };
            for (int j = 0; j < n && ok;) {
                if (j > 0) {
                    ok = products_before(j, two);
                    if (!ok) break;
                    if (busy) keep(j, m_ref, sum());
                    sum2 = 0;
                }
                for (const int end = min(n, j + CHUNK_SUM_STEPS); j < end; ++j) {
                    const int b = two ? t : 2 + (j & 1);  // S tile of this step
                    const int phase = two ? taken++ : (j & 1) ? taken_odd++ : taken_even++;
                    ok = __all_sync(FULL_MASK, mbar_wait_short(s_full(b), phase & 1));
                    if (!ok) break;
                    if (busy) {
                        umma::fence_after_sync();
                        const float2 ref = step_at(j);
                        const float by = step_scale(ref), moved = ref.y;
                        const uint32_t s_t = lane_tmem + (b & 1) * CHUNK_TILE;
                        const int seen = lim - (pc.kt0 + j) * CHUNK_TILE;  // columns this row may see
                        // with two tiles a step's S was committed after the P.V before, with one not
                        const uint32_t wait_o = two ? 0u : pv_step((j & 1) ^ 1);
                        const int phase_o = ((j & 1) ? taken_even : taken_odd) - 1;
                        const bool edge = __any_sync(FULL_MASK, seen < CHUNK_TILE);
                        // Two copies of the code, or one where the conversion's is there too, for the sake of the
                        // instruction cache: 24 requests of up to 512 queries, heads of 64, 48 us (52 with two);
                        // 500 queries over 130,500 tokens, heads of 128, fp16, 847 us (885 with two), but bf16
                        // 912 (861 with two).
                        if (Q8 && (D == 64 || KEYS_F16))
                            ok = softmax_step<M, D, SPLIT_P, Q8>(s_t, o_t, seen, edge, j > 0, by, moved, m_ref, sum2,
                                                                 p_full(b, 0), p_full(b, 1), wait_o, phase_o);
                        else if (edge)
                            ok = softmax_step<M, D, SPLIT_P, Q8>(s_t, o_t, seen, std::true_type(), j > 0, by, moved,
                                                                 m_ref, sum2, p_full(b, 0), p_full(b, 1), wait_o,
                                                                 phase_o);
                        else
                            ok = softmax_step<M, D, SPLIT_P, Q8>(s_t, o_t, seen, std::false_type(), j > 0, by, moved,
                                                                 m_ref, sum2, p_full(b, 0), p_full(b, 1), wait_o,
                                                                 phase_o);
                        if (!ok) break;
                    } else if (lane == 0) {  // rows of no query: whatever S left there
                        mbar_arrive(p_full(b, 0));
                        mbar_arrive(p_full(b, 1));
                    }
                }
            }
            if (!ok) break;
            steps += n;
            float l = sum();
            if (busy && n > CHUNK_SUM_STEPS) {
                ok = products_before(n, two, true);
                if (!ok) break;
                l = total(i, m_ref, l);
            }
            if (two) {
                p_clear = false;
                ++twos;
            }
            if (!hand_out(m_ref, l)) break;
        }
    }
    if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);

    // tensor memory goes back only after every warp is done with it
    umma::fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        umma::fence_after_sync();
        umma::dealloc(tmem, L::TMEM_COLS);
    }
}

// q seen as [T][Hq][D / 64][64]: a box is the G heads of one kv head for `tokens` tokens, one
// 128-byte column, landing as rows (token, head) of 128 bytes with the 128-byte swizzle.
template <typename T>
inline bool encode_query_map(CUtensorMap* map, const void* q, int T_, int Hq, int D, int G, int tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)(D / 64), (cuuint64_t)Hq, (cuuint64_t)T_};
    const cuuint64_t strides[3] = {128, (cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)G, (cuuint32_t)tokens};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, Mma<T>::TMA_TYPE, 4, const_cast<void*>(q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An 8-bit pool seen as [N * Hkv * B rows][D bytes]: boxes of 16 rows, as they lie.
inline bool encode_q8_map(CUtensorMap* map, const void* base, long long rows, int D) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D};
    const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)CHUNK_TOKENS};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool SPLIT_P, bool Q8>
cudaError_t launch_chunk_tds(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                             cudaStream_t stream) {
    constexpr int SMEM = ChunkSmem<D, Q8>::BYTES;
    const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
    const int G = p.group;
    CUtensorMap tq, tq32, tk, tv;
    if (!encode_query_map<T>(&tq, x.q, x.num_tokens, p.num_q_heads, D, G, 128 / G) ||
        !encode_query_map<T>(&tq32, x.q, x.num_tokens, p.num_q_heads, D, G, G <= 32 ? 32 / G : 1) ||
        !(Q8 ? encode_q8_map(&tk, x.k_pool, rows, D) : encode_pool_map<T>(&tk, x.k_pool, rows, D)) ||
        !(Q8 ? encode_q8_map(&tv, x.v_pool, rows, D) : encode_pool_map_3d<T>(&tv, x.v_pool, rows, D)))
        return cudaErrorNotSupported;
    auto kernel = chunk_attention_kernel<T, D, SPLIT_P, Q8>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> configured[64];  // per device; setting it twice is harmless
    if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    // nothing is launched before everything that may be refused
    e = launch_chunk_plan(plan, x.max_tiles, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x.ctas);
    cfg.blockDim = dim3(CHUNK_THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tq, tq32, tk, tv, p);
}

template <typename T, bool Q8>
cudaError_t launch_chunk_impl(const ChunkPlanParams& plan, const ChunkParams& p, const ChunkTensors& x,
                              cudaStream_t stream) {
    const bool f32_out = p.out_dtype == PKV_F32;
    if (p.head_dim == 64)
        return f32_out ? launch_chunk_tds<T, 64, true, Q8>(plan, p, x, stream)
                       : launch_chunk_tds<T, 64, false, Q8>(plan, p, x, stream);
    if (p.head_dim == 128)
        return f32_out ? launch_chunk_tds<T, 128, true, Q8>(plan, p, x, stream)
                       : launch_chunk_tds<T, 128, false, Q8>(plan, p, x, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
