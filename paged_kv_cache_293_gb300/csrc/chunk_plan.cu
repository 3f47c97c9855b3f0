// chunk_plan.cu -- the list of work of the chunk attention kernel (chunk.cuh), made on the
// device from the query starts and context lengths, and the merge of contexts it cut.
//
// A tile is up to 2 * (128 / G) consecutive queries of one request; a tile and a kv head are
// one item, whose steps are the 128-token stretches of the context its last query may see.
// An item is cut into several pieces along the context only where that shortens the whole:
// the cuts are tried for 1 to 32 pieces of the longest item, and the number with the
// smallest estimate taken, in steps of one CTA,
//   max(all steps / CTAs, min(rounds of pieces * (piece + F), all steps / CTAs + piece + F)) + merge
// (the first form in min() when pieces are alike, the second, list scheduling's bound, when
// they are not; F steps of fixed cost per piece).  Each cut item's pieces leave (m, l, o) per
// row, merged by log-sum-exp.  Lengths and the number of CTAs decide everything here, so the
// same batch is always cut, and summed, in the same way.
#include <cmath>

#include "pkv_common.cuh"

namespace pkv {

namespace {

constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ int4 add4(int4 a, int4 b) {
    return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

__device__ __forceinline__ int4 warp_scan4(int4 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int4 u = make_int4(__shfl_up_sync(FULL_MASK, v.x, o), __shfl_up_sync(FULL_MASK, v.y, o),
                                 __shfl_up_sync(FULL_MASK, v.z, o), __shfl_up_sync(FULL_MASK, v.w, o));
        if (lane >= o) v = add4(v, u);
    }
    return v;
}

// Inclusive sums over the CTA; `total` gets the sums over all threads.
__device__ __forceinline__ int4 block_scan4(int4 v, int4* warp_sums, int4* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_scan4(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = warp_scan4(warp_sums[lane], lane);
    __syncthreads();
    if (warp > 0) v = add4(v, warp_sums[warp - 1]);
    *total = warp_sums[31];
    __syncthreads();  // warp_sums is free again
    return v;
}

// Steps of a tile: 128-token stretches up to the last position its last query sees.
__device__ __forceinline__ int tile_steps(const int4& tile) {
    const int tok_end = tile.w + tile.z - 1;  // limit of the last query
    return tok_end > 0 ? (tok_end + CHUNK_TILE - 1) / CHUNK_TILE : 0;
}

}  // namespace

__global__ void __launch_bounds__(PLAN_THREADS) chunk_plan_kernel(const ChunkPlanParams p) {
    __shared__ int4 warp_sums[32];
    __shared__ int max_steps_s;
    __shared__ float est_s[32];
    // the attention kernel may set itself up meanwhile; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int QT = 2 * (128 / p.group);  // queries per tile
    if (tid == 0) {
        p.tile_start[0] = 0;
        max_steps_s = 0;
    }

    // ---- tiles of each request
    bool bad = false;
    int carry = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += PLAN_THREADS) {
        const int s = s0 + tid;
        int nt = 0;
        if (s < p.num_seqs) {
            const int a = p.query_start[s], b = p.query_start[s + 1];
            if (a < 0 || b < a || b > p.num_tokens)
                bad = true;
            else
                nt = (int)(((long long)b - a + QT - 1) / QT);
        }
        int4 total;
        const int4 v = block_scan4(make_int4(nt, 0, 0, 0), warp_sums, &total);
        // starts that do not ascend could sum past the list: such a batch is refused below
        if (s < p.num_seqs) p.tile_start[s + 1] = carry + v.x;
        carry += total.x;
        if (__syncthreads_or(bad)) {
            if (tid == 0) {
                set_error(p.err, PKV_DEVERR_POSITION);
                p.header[0] = p.header[1] = p.header[2] = p.header[3] = 0;
            }
            return;
        }
    }
    const int num_tiles = carry;

    // ---- one record per tile, the longest of a request first
    const long long cap = min((long long)p.max_blocks_per_seq * p.block_size, (long long)p.max_context_len);
    int steps = 0;
    for (int ti = tid; ti < num_tiles; ti += PLAN_THREADS) {
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {  // first request whose tiles end past ti
            const int mid = (lo + hi) >> 1;
            if (p.tile_start[mid + 1] > ti) hi = mid; else lo = mid + 1;
        }
        const int nq = p.query_start[lo + 1] - p.query_start[lo];
        int ctx = p.context_lens[lo];
        if (ctx < 0 || ctx > cap) {
            set_error(p.err, PKV_DEVERR_CONTEXT);
            ctx = ctx < 0 ? 0 : (int)cap;
        }
        const int j0 = (p.tile_start[lo + 1] - 1 - ti) * QT;
        const int4 tile = make_int4(lo, j0, min(QT, nq - j0), ctx - nq + 1 + j0);
        p.tiles[ti] = tile;
        steps = max(steps, tile_steps(tile));
    }
    atomicMax(&max_steps_s, steps);
    __syncthreads();
    const int max_steps = max_steps_s;

    // ---- pieces of the longest item: candidate k = warp + 1
    int cut = max_steps;  // steps per piece at most
    if (p.max_partial_rows > 0 && max_steps >= CHUNK_SPLIT_MIN) {
        const float F = 2.f, merge = 4.f;
        const int k = warp + 1, c = (max_steps + k - 1) / k;
        float all = 0.f;
        int n_pieces = 0, rows = 0, cuts = 0;
        for (int ti = lane; ti < num_tiles; ti += 32) {
            const int4 tile = p.tiles[ti];
            const int n = tile_steps(tile), pc = n > c ? (n + c - 1) / c : 1;
            all += (float)n + F * (float)pc;
            n_pieces += pc;
            if (pc > 1) {
                rows += pc * tile.z * p.group;
                cuts += pc;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            all += __shfl_xor_sync(FULL_MASK, all, o);
            n_pieces += __shfl_xor_sync(FULL_MASK, n_pieces, o);
            rows += __shfl_xor_sync(FULL_MASK, rows, o);
            cuts += __shfl_xor_sync(FULL_MASK, cuts, o);
        }
        if (lane == 0) {
            const float ctas = (float)p.num_sms, H = (float)p.num_kv_heads;
            const float mean = all * H / ctas;
            const float rounds = ceilf((float)n_pieces * H / ctas) * ((float)c + F);
            float est = fmaxf(mean, fminf(rounds, mean + (float)c + F)) + (k > 1 ? merge : 0.f);
            if (k > 1 && (c < 2 || (long long)rows * p.num_kv_heads > p.max_partial_rows ||
                          (long long)cuts * p.num_kv_heads > p.max_cut_pieces))
                est = INFINITY;
            est_s[warp] = est;
        }
        __syncthreads();
        int best = 0;
        for (int w = 1; w < 32; ++w)
            if (est_s[w] < est_s[best]) best = w;
        cut = (max_steps + best) / (best + 1);
    }

    // ---- the pieces, tile by tile, the heads of a tile behind one another
    int4 base = make_int4(0, 0, 0, 0);  // pieces, partial rows, cut items, their rows
    for (int t0 = 0; t0 < num_tiles; t0 += PLAN_THREADS) {
        const int ti = t0 + tid;
        int4 tile = make_int4(0, 0, 0, 0);
        int n = 0, pc = 0;
        if (ti < num_tiles) {
            tile = p.tiles[ti];
            n = tile_steps(tile);
            pc = n > cut ? (n + cut - 1) / cut : 1;
        }
        const int H = p.num_kv_heads, R = tile.z * p.group;
        const int4 mine = make_int4(H * pc, pc > 1 ? H * pc * R : 0, pc > 1 ? H : 0, pc > 1 ? H * R : 0);
        int4 total;
        const int4 v = block_scan4(mine, warp_sums, &total);
        if (pc > 0) {
            const int first = base.x + v.x - mine.x, row0 = base.y + v.y - mine.y;
            const int item0 = base.z + v.z - mine.z, mrow0 = base.w + v.w - mine.w;
            const int token = p.query_start[tile.x] + tile.y;
            for (int h = 0; h < H; ++h) {
                for (int r = 0; r < pc; ++r) {
                    ChunkPiece x;
                    x.token = token;
                    x.kv_head = h;
                    x.queries = tile.z;
                    x.lim0 = tile.w;
                    x.seq = tile.x;
                    x.kt0 = (int)((long long)n * r / pc);
                    x.kt1 = (int)((long long)n * (r + 1) / pc);
                    x.part_row = pc > 1 ? row0 + (h * pc + r) * R : -1;
                    p.pieces[first + h * pc + r] = x;
                }
                if (pc > 1) {
                    ChunkMerge m;
                    m.token = token;
                    m.kv_head = h;
                    m.rows = R;
                    m.parts = pc;
                    m.part_row = row0 + h * pc * R;
                    m.first = mrow0 + h * R;
                    m.pad0 = m.pad1 = 0;
                    p.merges[item0 + h] = m;
                }
            }
        }
        base = add4(base, total);
    }
    if (tid == 0) {
        p.header[0] = base.x;
        p.header[1] = base.z;
        p.header[2] = base.w;
        p.header[3] = p.ctas;  // pieces handed out: CTA i starts with piece i
    }
}

// One warp per row of a cut item: out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k over
// its pieces (at most 32: lane k holds piece k's weight).
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
    constexpr int V = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int rows = p.header[2], items = p.header[1];
    for (int g = blockIdx.x * 8 + (threadIdx.x >> 5); g < rows; g += gridDim.x * 8) {
        int lo = 0, hi = items - 1;
        while (lo < hi) {  // last item starting at or before g
            const int mid = (lo + hi + 1) >> 1;
            if (p.merges[mid].first <= g) lo = mid; else hi = mid - 1;
        }
        const ChunkMerge m = p.merges[lo];
        const int r = g - m.first;
        const long long row0 = (long long)m.part_row + r;
        float mk = -INFINITY, lk = 0.f;
        if (lane < m.parts) {
            mk = p.part_m[row0 + (long long)lane * m.rows];
            lk = p.part_l[row0 + (long long)lane * m.rows];
        }
        if (!(lk > 0.f)) mk = -INFINITY;
        float M = mk;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
        const float w = lk > 0.f ? fast_exp2(mk - M) : 0.f;
        float l = w * lk;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(FULL_MASK, l, o);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int k = 0; k < m.parts; ++k) {
            const float wk = __shfl_sync(FULL_MASK, w, k);
            const float* src = p.part_o + (row0 + (long long)k * m.rows) * D + lane * V;
            float v[V];
            if constexpr (V == 4) {
                const float4 x = *reinterpret_cast<const float4*>(src);
                v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(src);
                v[0] = x.x; v[1] = x.y;
            }
            // a piece that saw nothing for this row has weight 0 and zeros
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, v[i], acc[i]);
        }
        const size_t out = (((size_t)m.token + r / p.group) * p.num_q_heads + m.kv_head * p.group + r % p.group) * D +
                           lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) store_out(p.out, p.out_dtype, out + i, l > 0.f ? acc[i] / l : 0.f);
    }
}

cudaError_t launch_chunk_plan(const ChunkPlanParams& p, cudaStream_t stream) {
    chunk_plan_kernel<<<1, PLAN_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_chunk_merge(const ChunkParams& p, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, chunk_merge_kernel<64>, p)
                            : cudaLaunchKernelEx(&cfg, chunk_merge_kernel<128>, p);
}

}  // namespace pkv
