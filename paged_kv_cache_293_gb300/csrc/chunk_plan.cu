// chunk_plan.cu -- the list of work of the chunk attention kernel (chunk.cuh), made on the
// device from the query starts and context lengths, and the merge of contexts it cut.
//
// A tile is up to 2 * (128 / G) consecutive queries of one request; a tile and a kv head are
// one item, whose steps are the 128-token stretches of the context its last query may see.
// An item is cut into several pieces along the context only where that shortens the whole:
// the cuts are tried for 1 to 32 pieces of the longest item, and the number with the smallest
// estimate taken.  Pieces are handed out costliest first within each N (256 or 1024) tiles of the
// batch, so with no more tiles than that the end comes close to the larger of two lower bounds, in
// steps of one CTA with F steps of fixed cost per piece (a piece costs up to 6000 cycles beside its
// steps of 2400 to 2800):
//   all steps / CTAs,
//   ceil(pieces at least x long / CTAs) * x    for x = 4/4, 3/4, 2/4 and 1/4 of the longest
// plus the merge of the cut rows (a launch, and PARTIAL_ROWS_PER_STEP rows written and read
// again in the time of a step).  Each cut item's pieces leave (m, l, o) per row, merged by
// log-sum-exp.  Lengths and the number of CTAs decide everything here, so the same batch is
// always cut, and summed, in the same way.
#include <cmath>

#include "pkv_common.cuh"

namespace pkv {

namespace {

constexpr float PARTIAL_ROWS_PER_STEP = 7000.f;  // of 128 values: 1 KB each at about 5 TB/s in 1.45 us
constexpr int PIECE_STEPS = 2;       // F above
constexpr int COST_CLASSES = 16;
// What a piece costs, for its place in the list, in steps of two query tiles: a step of one tile
// waits for the HBM alone, and two tiles come with queries and outputs of up to 128 KB.  48
// requests, 70 % decoding, 40 / 40 heads: 245 us (256 by steps alone); 40 requests, 28 / 4 heads:
// 48.4 us (49.8); 24 requests of up to 512 queries, 16 / 4 heads of 64: 30.6 us (31.1).
constexpr float ONE_TILE_STEP = 0.7f, TWO_TILE_EXTRA = 1.5f;
constexpr int COUNT_MAX = 1 << 25;
// Items from which on no cuts are tried; the search took 2500 of the plan's 13,700 cycles for a
// mixed batch of 51 tiles and 40 heads.
constexpr float MANY_ITEMS = 3.f;

__device__ __forceinline__ int3 add3(int3 a, int3 b) { return make_int3(a.x + b.x, a.y + b.y, a.z + b.z); }

__device__ __forceinline__ int3 shfl3(int3 v, int from) {
    return make_int3(__shfl_sync(FULL_MASK, v.x, from), __shfl_sync(FULL_MASK, v.y, from),
                     __shfl_sync(FULL_MASK, v.z, from));
}

__device__ __forceinline__ int3 warp_scan3(int3 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int3 u = make_int3(__shfl_up_sync(FULL_MASK, v.x, o), __shfl_up_sync(FULL_MASK, v.y, o),
                                 __shfl_up_sync(FULL_MASK, v.z, o));
        if (lane >= o) v = add3(v, u);
    }
    return v;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL_MASK, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Inclusive sums over the CTA's N threads; `total` gets the sums over all of them.
template <int N>
__device__ __forceinline__ int3 block_scan3(int3 v, int3* warp_sums, int3* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_scan3(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    // every warp sums the warps before it itself: one barrier less
    const int3 w = warp_scan3(lane < N / 32 ? warp_sums[lane] : make_int3(0, 0, 0), lane);
    const int3 before = shfl3(w, warp > 0 ? warp - 1 : 0);
    if (warp > 0) v = add3(v, before);
    *total = shfl3(w, 31);
    __syncthreads();  // warp_sums is free again
    return v;
}

// The same for one value.
template <int N>
__device__ __forceinline__ int block_scan(int v, int3* warp_sums, int* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_scan(v, lane);
    if (lane == 31) warp_sums[warp].x = v;
    __syncthreads();
    const int w = warp_scan(lane < N / 32 ? warp_sums[lane].x : 0, lane);
    const int before = __shfl_sync(FULL_MASK, w, warp > 0 ? warp - 1 : 0);
    if (warp > 0) v += before;
    *total = __shfl_sync(FULL_MASK, w, 31);
    __syncthreads();
    return v;
}

// ceil(n / c) for 0 <= n < 2^24 steps, 1 <= c: rounded from 32-bit floats, then set right.
__device__ __forceinline__ int ceil_div_steps(int n, int c, float inv) {
    const int m = n + c - 1;
    int q = (int)((float)m * inv);
    const int r = m - q * c;
    return r < 0 ? q - 1 : r >= c ? q + 1 : q;
}

// Steps of a tile: 128-token stretches up to the last position its last query sees.
__device__ __forceinline__ int tile_steps(const int4& tile) {
    const int tok_end = tile.w + tile.z - 1;  // limit of the last query
    return tok_end > 0 ? (tok_end + CHUNK_TILE - 1) / CHUNK_TILE : 0;
}

}  // namespace

// One CTA: it is a chain of short dependent steps (load the lengths, sum, search, choose, sort,
// sum, write), N requests and N tiles at a time, whose arrays stay in shared memory when all
// of the batch fits into one round and go to the workspace when it does not.
template <int N>
__global__ void __launch_bounds__(N) chunk_plan_kernel(const ChunkPlanParams p) {
    __shared__ int3 warp_sums[32];
    __shared__ int max_steps_s, all_steps_s;
    __shared__ int sums_s[7][32];  // of each candidate
    __shared__ int start_s[N + 1], tile_start_s[N + 1], ctx_s[N];
    __shared__ int4 tiles_s[N];  // this round's tiles
    __shared__ int first_s[N];   // tiles before, by (class, warp)
    __shared__ int warp_pieces_s[32];
    __shared__ int3 base_s[N];   // pieces, partial rows, cut items before it
    // the attention kernel may set itself up meanwhile; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int QT = 2 * (128 / p.group);  // queries per tile
    const bool few = p.num_seqs <= N;
    int* tile_start = few ? tile_start_s : p.tile_start;
    const int* starts = few ? start_s : p.query_start;
    const int* ctxs = few ? ctx_s : p.context_lens;
    if (tid == 0) {
        tile_start[0] = 0;
        max_steps_s = all_steps_s = 0;
    }
    for (int i = tid; i < 7 * 32; i += N) sums_s[i >> 5][i & 31] = 0;

    // ---- tiles of each request
    int carry = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += N) {
        const int s = s0 + tid;
        int nt = 0;
        bool bad = false;
        if (s < p.num_seqs) {
            const int a = p.query_start[s], b = p.query_start[s + 1], c = p.context_lens[s];
            if (few) {
                start_s[s] = a;
                start_s[s + 1] = b;
                ctx_s[s] = c;
            }
            bad = a < 0 || b < a || b > p.num_tokens;
            if (!bad) nt = (int)(((long long)b - a + QT - 1) / QT);
        }
        // starts that do not ascend could sum past the list: such a batch is refused
        if (__syncthreads_or(bad)) {
            if (tid == 0) {
                set_error(p.err, PKV_DEVERR_POSITION);
                p.header[0] = p.header[1] = p.header[2] = 0;
            }
            return;
        }
        int total;
        const int v = block_scan<N>(nt, warp_sums, &total);
        if (s < p.num_seqs) tile_start[s + 1] = carry + v;
        carry += total;
    }
    const int num_tiles = carry;
    int4* tiles = num_tiles <= N ? tiles_s : p.tiles;
    __syncthreads();

    // ---- one record per tile, the longest of a request first
    const long long cap = min((long long)p.max_blocks_per_seq * p.block_size, (long long)p.max_context_len);
    int steps = 0, all_steps = 0;
    for (int ti = tid; ti < num_tiles; ti += N) {
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {  // first request whose tiles end past ti
            const int mid = (lo + hi) >> 1;
            if (tile_start[mid + 1] > ti) hi = mid; else lo = mid + 1;
        }
        const int nq = starts[lo + 1] - starts[lo];
        int ctx = ctxs[lo];
        if (ctx < 0 || ctx > cap) {
            set_error(p.err, PKV_DEVERR_CONTEXT);
            ctx = ctx < 0 ? 0 : (int)cap;
        }
        const int j0 = (tile_start[lo + 1] - 1 - ti) * QT;
        const int4 tile = make_int4(lo, j0, min(QT, nq - j0), ctx - nq + 1 + j0);
        tiles[ti] = tile;
        const int n = tile_steps(tile);
        steps = max(steps, n);
        all_steps = min(all_steps + n, COUNT_MAX / 32);
    }
    steps = __reduce_max_sync(FULL_MASK, steps);
    all_steps = (int)__reduce_add_sync(FULL_MASK, (unsigned)all_steps);
    if (lane == 0 && steps > 0) {
        atomicMax(&max_steps_s, steps);
        atomicAdd(&all_steps_s, all_steps);
    }
    __syncthreads();
    const int max_steps = max_steps_s;
    // each CTA's share of the steps is MANY_ITEMS of the longest item: the pieces handed out last
    // are short, and cutting could shorten nothing.  (Not so for a long context behind the first N
    // tiles: 512 tokens over 100,000 behind 1100 decoding requests 825 us, in front of them 741.)
    const bool many = (float)all_steps_s * (float)p.num_kv_heads >= MANY_ITEMS * (float)max_steps * (float)p.num_sms;

    // ---- pieces of the longest item: 32 candidates, some for each warp
    int cut = max(max_steps, 1);  // steps per piece at most
    if (p.max_partial_rows > 0 && max_steps >= CHUNK_SPLIT_MIN && !many) {
        // lane k - 1 of every warp: candidate k's steps per piece
        const int my_c = (max_steps + lane) / (lane + 1);
        const float my_inv = __fdividef(1.f, (float)my_c);
        int all = 0, rows = 0, cuts = 0, longer[4] = {0, 0, 0, 0};
        for (int ti = warp; ti < num_tiles; ti += N / 32) {
            const int4 tile = tiles[ti];
            const int n = tile_steps(tile), pc = n > my_c ? ceil_div_steps(n, my_c, my_inv) : 1;
            // (the largest batches would pass 32 bits; COUNT_MAX is more than any batch may cut,
            // and 32 warps of it still fit)
            all = min(all + n + PIECE_STEPS * pc, COUNT_MAX);
            if (pc > 1) {
                rows = min(rows + pc * tile.z * p.group, COUNT_MAX);
                cuts += pc;
            }
            // the longest of the tile's pieces counts for all of them
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (4 * (n + pc - 1) >= (4 - x) * my_c * pc) longer[x] += pc;
        }
        atomicAdd(&sums_s[0][lane], all);
        atomicAdd(&sums_s[1][lane], rows);
        atomicAdd(&sums_s[2][lane], cuts);
#pragma unroll
        for (int x = 0; x < 4; ++x) atomicAdd(&sums_s[3 + x][lane], longer[x]);
        __syncthreads();
        // lane k - 1 of every warp: candidate k's estimate
        const float H = (float)p.num_kv_heads, inv_sms = __fdividef(1.f, (float)p.num_sms);
        rows = sums_s[1][lane];
        cuts = sums_s[2][lane];
        float est = (float)sums_s[0][lane] * H * inv_sms;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            est = fmaxf(est, ceilf((float)sums_s[3 + x][lane] * H * inv_sms - 1e-4f) *
                                 (0.25f * (float)((4 - x) * my_c) + (float)PIECE_STEPS));
        if (lane > 0) {
            est += 3.f + (float)rows * H * (1.f / PARTIAL_ROWS_PER_STEP);
            if (my_c < 2 || (long long)rows * p.num_kv_heads > p.max_partial_rows ||
                (long long)cuts * p.num_kv_heads > p.max_cut_pieces)
                est = INFINITY;
        }
        // the smallest estimate, the fewest pieces among equals (estimates are not negative, so
        // their bits order like their values)
        const unsigned mine = __float_as_uint(est), least = __reduce_min_sync(FULL_MASK, mine);
        cut = __shfl_sync(FULL_MASK, my_c, __ffs(__ballot_sync(FULL_MASK, mine == least)) - 1);
    }

    // ---- the pieces, the heads of a tile behind one another
    const float inv_cut = 1.f / (float)cut;
    const int H = p.num_kv_heads;
    int* parts_s = ctx_s;          // of each tile: its pieces
    int* token_s = tile_start_s;   // and its first token (both arrays are done with)
    int3 base = make_int3(0, 0, 0);  // pieces, partial rows, cut items
    for (int t0 = 0; t0 < num_tiles; t0 += N) {
        const int ti = t0 + tid;
        const int live = min(N, num_tiles - t0);
        int4 tile = make_int4(0, 0, 0, 0);
        int pc = 0, len = 0;
        auto parts_of = [&](const int4& x) {
            const int n = tile_steps(x);
            return n > cut ? ceil_div_steps(n, cut, inv_cut) : 1;
        };
        if (ti < num_tiles) {
            tile = tiles[ti];
            pc = parts_of(tile);
            len = tile_steps(tile) / pc;
        }
        auto amounts = [&] {
            return make_int3(H * pc, pc > 1 ? H * pc * tile.z * p.group : 0, pc > 1 ? H : 0);
        };
        int3 mine = amounts(), total;
        const int warp_pieces = (int)__reduce_add_sync(FULL_MASK, (unsigned)mine.x);
        if (lane == 0) warp_pieces_s[warp] = warp_pieces;
        __syncthreads();
        if (__reduce_add_sync(FULL_MASK, (unsigned)(lane < N / 32 ? warp_pieces_s[lane] : 0)) > (unsigned)p.ctas) {
            // costliest pieces first: a counting sort of the round's tiles by classes of cost, in
            // tile order within a class
            const float most = (float)cut + TWO_TILE_EXTRA;
            const float cost = tile.z > QT / 2 ? (float)len + TWO_TILE_EXTRA : ONE_TILE_STEP * (float)len;
            const int cls = ti < num_tiles ? min(COST_CLASSES - 1, (int)((most - cost) * (COST_CLASSES / most)))
                                           : COST_CLASSES;  // no tile: behind the others
            const unsigned same = __match_any_sync(FULL_MASK, cls);
            const int before = __popc(same & ((1u << lane) - 1u));
            // counts by (class, warp), then their sums: entry c * W + w is class c of warp w
            constexpr int W = N / 32, COUNTS = COST_CLASSES * W;
            static_assert(COUNTS <= N, "one count per thread");
            if (lane < COST_CLASSES) first_s[lane * W + warp] = 0;
            __syncwarp();
            if (before == 0 && cls < COST_CLASSES) first_s[cls * W + warp] = __popc(same);
            __syncthreads();
            const int count = tid < COUNTS ? first_s[tid] : 0;
            int all_tiles;
            const int upto = block_scan<N>(count, warp_sums, &all_tiles);
            if (tid < COUNTS) first_s[tid] = upto - count;
            __syncthreads();
            if (cls < COST_CLASSES) tiles_s[first_s[cls * W + warp] + before] = tile;
            __syncthreads();
            if (ti < num_tiles) {
                tile = tiles_s[tid];
                pc = parts_of(tile);
            }
            mine = amounts();
        } else if (ti < num_tiles) {
            tiles_s[tid] = tile;
        }
        const int3 v = block_scan3<N>(mine, warp_sums, &total);
        parts_s[tid] = pc;
        token_s[tid] = ti < num_tiles ? starts[tile.x] + tile.y : 0;
        base_s[tid] = make_int3(base.x + v.x - mine.x, base.y + v.y - mine.y, base.z + v.z - mine.z);
        __syncthreads();
        // `lanes` lanes write a tile's pieces
        const int lanes = H >= 32 ? 32 : 1 << (32 - __clz(max(H - 1, 0)));  // H rounded up to a power of two
#pragma unroll 1
        for (int k = tid / lanes; k < live; k += N / lanes) {
            const int4 x = tiles_s[k];
            const int3 at = base_s[k];
            const int n = tile_steps(x), parts = parts_s[k], token = token_s[k], rows = x.z * p.group;
            int4* out = reinterpret_cast<int4*>(p.pieces + at.x);
            if (parts == 1) {
#pragma unroll 1
                for (int h = tid & (lanes - 1); h < H; h += lanes) {
                    out[2 * h] = make_int4(token, h, x.z, x.w);
                    out[2 * h + 1] = make_int4(x.x, 0, n, -1);
                }
                continue;
            }
#pragma unroll 1
            for (int e = tid & (lanes - 1); e < H * parts; e += lanes) {
                const int h = e / parts, r = e - h * parts;
                // (at most 2^24 steps and 32 parts)
                const int kt0 = (int)((unsigned)n * (unsigned)r / (unsigned)parts);
                const int kt1 = (int)((unsigned)n * (unsigned)(r + 1) / (unsigned)parts);
                const int part_row = at.y + e * rows;
                out[2 * e] = make_int4(token, h, x.z, x.w);
                out[2 * e + 1] = make_int4(x.x, kt0, kt1, part_row);
                if (r == 0) {
                    ChunkMerge m;
                    m.token = token;
                    m.kv_head = h;
                    m.rows = rows;
                    m.parts = parts;
                    m.part_row = part_row;
                    m.lim0 = x.w;
                    m.pad0 = m.pad1 = 0;
                    p.merges[at.z + h] = m;
                }
            }
        }
        base = add3(base, total);
        __syncthreads();
    }
    if (tid == 0) {
        p.header[0] = base.x;
        p.header[1] = base.z;
        p.header[2] = p.ctas;  // pieces handed out: CTA i starts with piece i
    }
}

// One warp per row of a cut item: out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k over
// its pieces (at most 32: lane k holds piece k's weight).  A CTA takes every n-th group of eight
// rows of one item, where n CTAs share it, so that a row's way is three loads behind one another:
// counts, item, results.
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
    constexpr int V = D / 32, AHEAD = 4;  // results loaded before their weights are known
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int items = p.header[1];
    if (items == 0) return;
    const int share = max(1, (int)gridDim.x / items);  // CTAs of an item
    if ((int)blockIdx.x >= items * share) return;
    for (int item = (int)blockIdx.x % items; item < items; item += (int)gridDim.x) {
        const ChunkMerge m = p.merges[item];
        for (int r = (int)blockIdx.x / items * 8 + warp; r < m.rows; r += share * 8) {
            const long long row0 = (long long)m.part_row + r;
            const float* src = p.part_o + row0 * D + lane * V;
            const long long apart = (long long)m.rows * D;
            auto load = [&](float (&v)[V], int k) {
                if constexpr (V == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src + k * apart);
                    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(src + k * apart);
                    v[0] = x.x; v[1] = x.y;
                }
            };
            float v[AHEAD][V];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k < m.parts) load(v[k], k);
            float mk = -INFINITY, lk = 0.f;
            if (lane < m.parts) {
                mk = p.part_m[row0 + (long long)lane * m.rows];
                lk = p.part_l[row0 + (long long)lane * m.rows];
            }
            if (lk == 0.f) mk = -INFINITY;  // (a NaN goes on)
            float M = mk;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
            const float w = lk == 0.f ? 0.f : fast_exp2(mk - M);
            float l = w * lk;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(FULL_MASK, l, o);
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            // (a piece that saw nothing for this row has weight 0 and zeros)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float wk = __shfl_sync(FULL_MASK, w, k);
                if (k < m.parts) {
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, v[k][i], acc[i]);
                }
            }
#pragma unroll 4
            for (int k = AHEAD; k < m.parts; ++k) {
                const float wk = __shfl_sync(FULL_MASK, w, k);
                float x[V];
                load(x, k);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, x[i], acc[i]);
            }
            const size_t out =
                (((size_t)m.token + r / p.group) * p.num_q_heads + m.kv_head * p.group + r % p.group) * D + lane * V;
#pragma unroll
            for (int i = 0; i < V; ++i)
                store_out(p.out, p.out_dtype, out + i, m.lim0 + r / p.group > 0 ? acc[i] / l : 0.f);
        }
    }
}

cudaError_t launch_chunk_plan(const ChunkPlanParams& p, int64_t max_tiles, cudaStream_t stream) {
    // few requests and tiles: fewer warps, whose sums and barriers are shorter (six short requests
    // 16.0 us in all, 17.8 with 1024 threads)
    const bool few = p.num_seqs <= 256 && max_tiles <= 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(few ? 256 : 1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, chunk_plan_kernel<256>, p)
               : cudaLaunchKernelEx(&cfg, chunk_plan_kernel<1024>, p);
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
