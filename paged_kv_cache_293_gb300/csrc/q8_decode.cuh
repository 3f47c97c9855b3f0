// q8_decode.cuh -- decode attention over a paged cache held in 8 bits ("What Is vLLM", section
// "How does PagedAttention work?": every cached position is found through the block table and
// read from the physical block holding it).
//
// For a query row q, pages b with scales a_b (keys) and c_b (values) and e4m3 values K, V:
//   s_t = scale a_b (q . K_t),   out = sum_b c_b sum_t e^(s_t - m) V_t / sum_t e^(s_t - m)
// HBM bound: a token of a kv head is 2 D bytes, read once for the G heads that share it, so the
// work per byte is twice that of a 16-bit cache and the kernel is laid out to need few
// instructions a byte.  Both products run on mma.sync.m16n8k16 in fp16, which holds every e4m3
// value: scores^T [16 tokens x 8] = K . Q^T and O^T [D x 8] = V^T . P^T, the 8 columns being the
// (query, head) pairs of one kv head.  Each warp brings 16 tokens at a time into a ring of its own by
// cp.async (a page's 16 tokens are D / 8 rows of 128 bytes, their 16-byte columns turned so that
// the reads below meet no bank twice) and takes the operands from there as they lie:
//   K  lane (g, c) = (lane / 4, lane % 4) reads D / 4 bytes in a row of tokens g and g + 8; the order of
//      a product's D terms is free, so the 4 values of a word are a lane's terms of one k step
//      (and Q is laid out alike);
//   V  lane (g, c) reads the D / 8 bytes from g D / 8 on of tokens 2c, 2c + 1, 2c + 8, 2c + 9: the
//      four tokens that its part of a k step takes, whose bytes one prmt a pair brings together.
// No barrier in the loop: a warp's lanes wait for their own copies, then for one another.  A page's
// scale a_b goes into the factor that its scores are multiplied with anyway, and c_b into the sum of its
// O into the row's, in 32 bits.
// Each row's reference follows its maximum and is raised only where a score exceeds it by more
// than 15 in base 2 (it is set 7 below the maximum), so no lane asks the others for theirs but then.
// P enters its product in fp16 (weights from 2^-21 of the largest on with 11 bits, none off by more
// than 2^-32 of it), and with a 32-bit output in two parts.
// Measured: 128 requests of ~600 tokens, 40 heads, fp16: 123 us, 6.2 TB/s (233 from 16 bits); 8 contexts of
// ~80000 tokens, 32 / 8 heads, bf16: 250 us with the merge, 6.4 TB/s (457).  What got it there, for the first:
// operands loaded straight to registers 162 us, too few bytes on their way at 12 warps of 158 registers;
// this ring with three stages and four CTAs per SM 122 us (two stages 128, three CTAs with four 127, eight
// warps a CTA 136).  Few requests (4 of ~700 tokens: 7.1 us) are a chain of dependent loads (length,
// table, scale and page), three or four steps and the cluster's meeting, which
// replaced a merge kernel (9.7 us).
#pragma once

#include <cfloat>
#include <climits>

#include "decode_mma.cuh"
#include "q8.cuh"

namespace pkv {

constexpr int Q8_WARPS = 4;
constexpr float Q8_BELOW = 7.f, Q8_RAISE = 15.f;

// 16 bytes global -> shared past L1, asynchronously; groups of copies and the wait for all but N.
__device__ __forceinline__ void cp_async16_stream(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_but() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The 8 x 8 matrix of 16-bit values whose row lane / 4 this lane has a pair of, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// All ones in the bytes of four e4m3 values that are NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

template <typename T> __device__ __forceinline__ float2 pair_to_floats(uint32_t w);
template <> __device__ __forceinline__ float2 pair_to_floats<__half>(uint32_t w) { return float2_of_f16x2(w); }
template <> __device__ __forceinline__ float2 pair_to_floats<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 16 tokens of one pool in shared memory: rows of 128 bytes, one token (D = 128) or two (D = 64), the
// 16-byte column j of row r at column j ^ turn(r).
template <int D>
struct Q8Tile {
    static constexpr int BYTES = CHUNK_TOKENS * D, COLUMNS = BYTES / 16;
    __device__ __forceinline__ static int at(int row, int col) {
        return row * 128 + ((col ^ (D == 128 ? row & 7 : 2 * (row & 3))) << 4);
    }
    // elements 4 w .. 4 w + 3 of token t
    __device__ __forceinline__ static int at_word(int t, int w) {
        return (D == 128 ? at(t, w >> 2) : at(t >> 1, 4 * (t & 1) + (w >> 2))) + 4 * (w & 3);
    }
    // word w of a lane's part of token t: of a key, bytes c D / 4 + 4 w .. + 3
    __device__ __forceinline__ static void key(const unsigned char* tile, int t, int c, uint32_t (&k)[D / 16]) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int col = D == 128 ? 2 * c + i : 4 * (t & 1) + c;
            const uint4 w = *reinterpret_cast<const uint4*>(tile + at(D == 128 ? t : t >> 1, col));
            k[4 * i] = w.x; k[4 * i + 1] = w.y; k[4 * i + 2] = w.z; k[4 * i + 3] = w.w;
        }
    }
    // of a value, bytes g D / 8 + 4 w .. + 3
    __device__ __forceinline__ static void value(const unsigned char* tile, int t, int g, uint32_t (&v)[D / 32]) {
        if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(tile + at(t, g));
            v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(tile + at(t >> 1, 4 * (t & 1) + (g >> 1)) + 8 * (g & 1));
            v[0] = w.x; v[1] = w.y;
        }
    }
};

// Stages of a warp's ring, and CTAs per SM that the registers are held to.  The rings' memory serves the warps'
// results afterwards, and one more row of them.
constexpr int Q8_STAGES = 3, Q8_CTAS = 4;
template <int D, int NT>
constexpr int q8_smem_bytes() {
    const int rings = Q8_WARPS * Q8_STAGES * 2 * Q8Tile<D>::BYTES, results = (Q8_WARPS + 1) * 8 * NT * (D + 2) * 4;
    return rings > results ? rings : results;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit value that CTA `rank` of the cluster has at this CTA's shared-memory address a.
__device__ __forceinline__ float load_from_cta(uint32_t a, uint32_t rank) {
    uint32_t there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
}

// NT: 8-column tiles of the products, 1 or 2.  SEVERAL: queries a sequence, which do not see the same tokens
// (an instance of its own: the code for values that some of them see, in a kernel of one query, cost 128 requests
// of ~600 tokens 2 % and 64 of ~500 7 %).
template <typename T, int D, int NT, bool SPLIT_P, bool SEVERAL>
__global__ void __launch_bounds__(Q8_WARPS * 32, NT * D > 128 ? Q8_CTAS - 1 : Q8_CTAS)
q8_decode_kernel(const Q8DecodeParams p) {
    constexpr int KS = D / 16, NW = Q8_WARPS, NS = Q8_STAGES, COLS = 8 * NT;
    using Tile = Q8Tile<D>;
    extern __shared__ __align__(128) unsigned char q8_smem[];
    __shared__ float2 stage_scale[NW][NS];
    __shared__ uint32_t nan_marks[SEVERAL ? NW : 1][COLS][D / 32];  // elements that are NaN besides, a bit each
    bool marked = false;                                           // this warp has made some
    // [NW], and one for the CTA's result in a cluster, once the rings are done with
    float(*red)[COLS][D + 2] = reinterpret_cast<float(*)[COLS][D + 2]>(q8_smem);
    const int Hkv = p.num_kv_heads, Hq = p.num_q_heads, G = Hq / Hkv, NQ = p.num_queries, B = p.block_size;
    const int kvh = blockIdx.x % Hkv, col0 = (blockIdx.x / Hkv) * COLS, s = blockIdx.y;
    const int part = gridDim.z - 1 - blockIdx.z;  // the last pieces, which few contexts reach, first
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int ncols = min(COLS, NQ * G - col0);
    // column n: query (col0 + n) / G, head (col0 + n) % G of the kv head
    auto row_of = [&](int n) -> size_t {
        return ((size_t)s * NQ + (col0 + n) / G) * Hq + kvh * G + (col0 + n) % G;
    };

    int ctx = p.context_lens[s];
    const long long table = (long long)p.max_blocks_per_seq * B;
    const int cap = (int)(table < p.max_context_len ? table : p.max_context_len);
    if (ctx < 0 || ctx > cap) {
        if (threadIdx.x == 0 && part == 0 && blockIdx.x == 0) set_error(p.err, PKV_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : cap;
    }
    const int P = p.partition_size, n_parts = (ctx + P - 1) / P, tok0 = part * P;
    if (!p.clustered && part > 0 && tok0 >= ctx) return;
    const bool direct = n_parts <= 1;
    const int tok_end = min(ctx, tok0 + P);
    const int n_chunks = max(tok_end - tok0 + CHUNK_TOKENS - 1, 0) / CHUNK_TOKENS;
    const int n_my = warp < n_chunks ? (n_chunks - warp + NW - 1) / NW : 0;

    // this warp's pages, 32 steps at a time: lane i has the page of step i, and its scales
    const int32_t* bt_row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const int shift = B == 32 ? 5 : 4;  // B is 16 or 32
    auto token_of = [&](int i) { return tok0 + (warp + NW * i) * CHUNK_TOKENS; };
    int page = -1;
    float ka = 0.f, va = 0.f;
    auto look_up = [&](int i) {
        page = -1;
        if (i >= n_my) return;
        const int phys = __ldg(bt_row + (token_of(i) >> shift));
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            set_error(p.err, PKV_DEVERR_BLOCK_ID);
            return;
        }
        page = phys;
        const size_t at = (size_t)phys * Hkv + kvh;
        ka = __ldg(p.k_scale + at);
        va = __ldg(p.v_scale + at);
    };
    unsigned char* const ring = q8_smem + warp * NS * 2 * Tile::BYTES;
    unsigned there = 0;  // stages that hold a page; bit 31: one did
    int first = INT_MAX;  // (several queries) from where on
    auto issue = [&](int i) {
        if (i < n_my) {
            if ((i & 31) == 0) look_up(i + lane);
            const int phys = __shfl_sync(FULL_MASK, page, i & 31), st = i % NS;
            const float a_b = __shfl_sync(FULL_MASK, ka, i & 31), c_b = __shfl_sync(FULL_MASK, va, i & 31);
            there = phys >= 0 ? there | (1u << st | 1u << 31) : there & ~(1u << st);
            if (SEVERAL && phys >= 0) first = min(first, token_of(i));
            if (lane == 0) stage_scale[warp][st] = make_float2(a_b, c_b);
            if (phys >= 0) {
                const size_t at = ((((size_t)phys * Hkv + kvh) << shift) + (token_of(i) & (B - 1))) * D;
                const uint32_t dst = smem_addr(ring + st * 2 * Tile::BYTES);
#pragma unroll
                for (int j = lane; j < Tile::COLUMNS; j += 32) {
                    const uint32_t to = dst + Tile::at(j >> 3, j & 7);
                    cp_async16_stream(to, p.k_pool + at + 16 * j);
                    cp_async16_stream(to + Tile::BYTES, p.v_pool + at + 16 * j);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) issue(i);

    // Q^T: column g's terms c D / 4 + 4 w .. + 3 for k step w, in fp16.  bf16 rows are
    // scaled by the power of two that brings their largest below 2^14, which keeps their bits.
    uint32_t qb[NT][KS][2];
    // this lane's columns of the scores on: 8 nt + 2 c and the next one, of tokens g and g + 8
    float f[NT][2], m_ref[NT][2], l[NT][2];
    int lim[NT][2], lim_all = ctx;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = 8 * nt + g;
        float q_inv = 1.f;  // of column g
        const T* src = static_cast<const T*>(p.q) + row_of(col < ncols ? col : 0) * D;
        uint32_t w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + c * (D / 4)) + i);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 v = pair_to_floats<T>(w[i]);
                top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
            top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
            top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
            // top < 2^(e + 1): times 2^(13 - e); rows below 2^-80 keep that factor
            const int e = max((__float_as_int(top) >> 23) - 127, -80);
            const float mul = __int_as_float((13 - e + 127) << 23);
            q_inv = __int_as_float((e - 13 + 127) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 v = pair_to_floats<T>(w[i]);
                w[i] = Mma<__half>::pack(v.x * mul, v.y * mul);
            }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) qb[nt][ks][h] = col < ncols ? w[2 * ks + h] : 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = 8 * nt + 2 * c + h;
            f[nt][h] = p.scale_log2 * __shfl_sync(FULL_MASK, q_inv, 4 * (2 * c + h));
            m_ref[nt][h] = -INFINITY;
            l[nt][h] = 0.f;
            lim[nt][h] = n < ncols ? ctx - NQ + 1 + (col0 + n) / G : ctx;  // positions below are seen
            lim_all = min(lim_all, lim[nt][h]);
        }
    }
    float o[NT][KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < KS; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;

    for (int i = 0; i < n_my; ++i) {
        const int t0 = token_of(i), st = i % NS;
        cp_async_wait_but<NS - 2>();
        __syncwarp();  // every lane's copies of this stage are there, and all are done with the stage before
        issue(i + NS - 1);
        const unsigned char* const k_tile = ring + st * 2 * Tile::BYTES;
        const float2 scales = stage_scale[warp][st];
        const float a_b = scales.x, c_b = scales.y;
        const bool here = (there >> st) & 1;

        float pr[NT][4];  // scores, then weights: token g + 8 (j / 2), column 8 nt + 2 c + j % 2
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) pr[nt][0] = pr[nt][1] = pr[nt][2] = pr[nt][3] = 0.f;
        {
            uint32_t k0[KS], k1[KS];
            Tile::key(k_tile, g, c, k0);
            Tile::key(k_tile, g + 8, c, k1);
            float odd[NT][4];  // two sums side by side: a product waits for the one before the last
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) odd[nt][0] = odd[nt][1] = odd[nt][2] = odd[nt][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a0, a1, a2, a3;
                f16x4_of_e4m3x4(k0[ks], a0, a2);
                f16x4_of_e4m3x4(k1[ks], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    Mma<__half>::run(ks & 1 ? odd[nt] : pr[nt], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) pr[nt][j] += odd[nt][j];
        }
        uint32_t v[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) Tile::value(k_tile + Tile::BYTES, 2 * c + (r & 1) + 8 * (r >> 1), g, v[r]);

        // in base 2
        float over = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) pr[nt][j] *= f[nt][j & 1] * a_b;
        if (!here || t0 + CHUNK_TOKENS > tok_end || __any_sync(FULL_MASK, t0 + CHUNK_TOKENS > lim_all)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = t0 + g + 8 * (j >> 1);
                    if (!here || t >= tok_end || t >= lim[nt][j & 1]) pr[nt][j] = -INFINITY;
                }
            // values of tokens that no row sees may be anything, and 0 * NaN is not 0
            const int seen = here ? tok_end - t0 : 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (2 * c + (r & 1) + 8 * (r >> 1) >= seen) {
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) v[r][w] = 0u;
                }
            if constexpr (SEVERAL) {
                // nor is it for a query that does not see a token which later ones do
                uint32_t nan = 0u;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) nan |= nan_codes(v[r][w]);
                if (__any_sync(FULL_MASK, nan != 0u)) {
                    // NaN values become zeros, noted for the columns that see them
                    if (!marked)
                        for (int x = lane; x < COLS * (D / 32); x += 32) (&nan_marks[warp][0][0])[x] = 0u;
                    marked = true;
                    __syncwarp();
                    unsigned char* const v_tile = ring + st * 2 * Tile::BYTES + Tile::BYTES;
#pragma unroll 1
                    for (int x = lane; x < CHUNK_TOKENS * (D / 4); x += 32) {
                        const int t = x / (D / 4), w = x % (D / 4);
                        uint32_t* const at = reinterpret_cast<uint32_t*>(v_tile + Tile::at_word(t, w));
                        const uint32_t codes = t < seen ? nan_codes(*at) : 0xffffffffu;
                        *at &= ~codes;
                        if (codes == 0u || t >= seen) continue;
                        // (a bit a byte)
                        const uint32_t bits = ((codes & 0x08040201u) * 0x01010101u >> 24) << (4 * w % 32);
                        for (int n = 0; n < ncols; ++n)
                            if (t0 + t < ctx - NQ + 1 + (col0 + n) / G)
                                atomicOr(&nan_marks[warp][n][w / 8], bits);
                    }
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 4; ++r) Tile::value(v_tile, 2 * c + (r & 1) + 8 * (r >> 1), g, v[r]);
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) over = fmaxf(over, pr[nt][j] - m_ref[nt][j & 1]);
        if (__any_sync(FULL_MASK, over > Q8_RAISE)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = fmaxf(pr[nt][h], pr[nt][h + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, d));
                    const float ref = top - m_ref[nt][h] > Q8_RAISE ? top - Q8_BELOW : m_ref[nt][h];
                    alpha[h] = ref == m_ref[nt][h] ? 1.f : fast_exp2(m_ref[nt][h] - ref);
                    m_ref[nt][h] = ref;
                    l[nt][h] *= alpha[h];
                }
#pragma unroll
                for (int d = 0; d < KS; ++d) {
                    o[nt][d][0] *= alpha[0]; o[nt][d][1] *= alpha[1];
                    o[nt][d][2] *= alpha[0]; o[nt][d][3] *= alpha[1];
                }
            }
        }
        uint32_t pb[NT][2], rb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float(&x)[4] = pr[nt];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m_ref[nt][h] == -INFINITY ? 0.f : m_ref[nt][h];
                x[h] = fast_exp2(x[h] - ref);
                x[h + 2] = fast_exp2(x[h + 2] - ref);
                l[nt][h] += x[h] + x[h + 2];
            }
            pb[nt][0] = transpose8x8(Mma<__half>::pack(x[0], x[1]));
            pb[nt][1] = transpose8x8(Mma<__half>::pack(x[2], x[3]));
            if (SPLIT_P) {
                float rem[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) rem[j] = x[j] - Mma<__half>::round_trip(x[j]);
                rb[nt][0] = transpose8x8(Mma<__half>::pack(rem[0], rem[1]));
                rb[nt][1] = transpose8x8(Mma<__half>::pack(rem[2], rem[3]));
            }
        }
        // rows of O^T's tile 2 w + h: elements g D / 8 + 4 w + 2 h and the next one
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a0, a1, a2, a3;
                f16x4_of_e4m3x4(__byte_perm(v[0][w], v[1][w], h == 0 ? 0x5140 : 0x7362), a0, a1);
                f16x4_of_e4m3x4(__byte_perm(v[2][w], v[3][w], h == 0 ? 0x5140 : 0x7362), a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    Mma<__half>::run(sum, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    if (SPLIT_P) Mma<__half>::run(sum, a0, a1, a2, a3, rb[nt][0], rb[nt][1]);
                    float(&od)[4] = o[nt][2 * w + h];
#pragma unroll
                    for (int j = 0; j < 4; ++j) od[j] = fmaf(sum[j], c_b, od[j]);
                }
            }
    }
    __syncthreads();  // the rings are done with (no copy is in flight: the last waits were for all that were issued)

    // ---- the warps' results together
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = l[nt][h];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
            float* r = red[warp][8 * nt + 2 * c + h];
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                r[g * (D / 8) + 2 * i] = o[nt][i][h];
                r[g * (D / 8) + 2 * i + 1] = o[nt][i][h + 2];
            }
            if (g == 0) {
                // (-inf: a row that sees no page; one whose scores are all -inf does)
                const bool sees = SEVERAL ? first < lim[nt][h] : there >> 31 != 0u;
                r[D] = sees ? fmaxf(m_ref[nt][h], -FLT_MAX) : m_ref[nt][h];
                r[D + 1] = sum;
            }
            if (SEVERAL && marked) {
                constexpr int EACH = D / 8;  // of this lane's elements
                uint32_t nan = nan_marks[warp][8 * nt + 2 * c + h][g * EACH / 32] >> (g * EACH % 32);
                for (nan &= (1u << EACH) - 1; nan != 0u; nan &= nan - 1)
                    r[g * EACH + __ffs(nan) - 1] = __int_as_float(0x7fffffff);
            }
        }
    __syncthreads();
    // zero for a row that sees nothing; a NaN or a sum of no weight is the result
    auto finish = [&](int n, int d, float M, float O, float L) {
        store_out(p.out, p.out_dtype, row_of(n) * D + d, M == -INFINITY ? 0.f : O / L);
    };
    for (int i = threadIdx.x; i < ncols * D; i += NW * 32) {
        const int n = i / D, d = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, red[w][n][D]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float by = fast_exp2(red[w][n][D] - ref);
            L = fmaf(red[w][n][D + 1], by, L);
            O = fmaf(red[w][n][d], by, O);
        }
        if (p.clustered) {
            red[NW][n][d] = O;
            if (d == 0) {
                red[NW][n][D] = M;
                red[NW][n][D + 1] = L;
            }
        } else if (direct) {
            finish(n, d, M, O, L);
        } else {
            const size_t at_part = row_of(n) * p.max_parts + part;
            p.part_o[at_part * D + d] = O;
            if (d == 0) {
                p.part_m[at_part] = M;
                p.part_l[at_part] = L;
            }
        }
    }
    if (p.clustered) {
        // the pieces of a context, a CTA each, from one another's shared memory: CTA r takes every
        // gridDim.z-th of the rows' elements
        cluster_sync();
        const int parts = gridDim.z;
        for (int i = blockIdx.z * (NW * 32) + threadIdx.x; i < ncols * D; i += parts * (NW * 32)) {
            const int n = i / D, d = i % D;
            const uint32_t at = smem_addr(&red[NW][n][0]);
            float m[Q8_CLUSTER], M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int k = 0; k < Q8_CLUSTER; ++k) {
                m[k] = k < parts ? load_from_cta(at + D * 4, k) : -INFINITY;
                M = fmaxf(M, m[k]);
            }
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < Q8_CLUSTER; ++k)
                if (k < parts) {
                    const float by = fast_exp2(m[k] - ref);
                    L = fmaf(load_from_cta(at + (D + 1) * 4, k), by, L);
                    O = fmaf(load_from_cta(at + d * 4, k), by, O);
                }
            finish(n, d, M, O, L);
        }
        cluster_sync();  // no CTA ends while others read its shared memory
    }
}

template <typename T, int D, int NT, bool SPLIT_P, bool SEVERAL>
cudaError_t launch_q8_decode_tdnsq(const Q8DecodeParams& p, cudaStream_t stream) {
    constexpr int SMEM = q8_smem_bytes<D, NT>();
    auto kernel = q8_decode_kernel<T, D, NT, SPLIT_P, SEVERAL>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> configured[64];  // per device; setting it twice is harmless
    if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    const int cols = p.num_queries * (p.num_q_heads / p.num_kv_heads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.num_kv_heads * ((cols + 8 * NT - 1) / (8 * NT))), (unsigned)p.num_seqs,
                       (unsigned)p.max_parts);
    cfg.blockDim = dim3(Q8_WARPS * 32);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)p.max_parts;
    cfg.attrs = attr;
    cfg.numAttrs = p.clustered ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int D, int NT, bool SPLIT_P>
cudaError_t launch_q8_decode_tdns(const Q8DecodeParams& p, cudaStream_t stream) {
    return p.num_queries > 1 ? launch_q8_decode_tdnsq<T, D, NT, SPLIT_P, true>(p, stream)
                             : launch_q8_decode_tdnsq<T, D, NT, SPLIT_P, false>(p, stream);
}

template <typename T, int D>
cudaError_t launch_q8_decode_td(const Q8DecodeParams& p, cudaStream_t stream) {
    const bool split = p.out_dtype == PKV_F32;
    if (p.column_tiles == 1)
        return split ? launch_q8_decode_tdns<T, D, 1, true>(p, stream) : launch_q8_decode_tdns<T, D, 1, false>(p, stream);
    return split ? launch_q8_decode_tdns<T, D, 2, true>(p, stream) : launch_q8_decode_tdns<T, D, 2, false>(p, stream);
}

template <typename T>
cudaError_t launch_q8_decode_impl(const Q8DecodeParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch_q8_decode_td<T, 64>(p, stream);
    if (head_dim == 128) return launch_q8_decode_td<T, 128>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
