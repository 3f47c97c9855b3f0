// batch.cu -- one ragged step's block tables, starts, positions and slots from the request
// lengths alone ("What Is vLLM", section "How does PagedAttention work?": blocks are
// allocated on demand; section "What is continuous batching in vLLM?": every step carries
// requests at different stages, so their lengths differ).
//
// With past_s cached and new_s arriving tokens of request s and B tokens per block,
//   need_s = ceil((past_s + new_s) / B) - ceil(past_s / B),  upto_s = need_0 + ... + need_s,
// a request is served when need_s = 0 or upto_s <= free: the free blocks go to the requests
// in order, and a request's j-th fresh block is the (upto_s - need_s + j)-th from the top of
// the free stack -- the ids a host loop popping them one by one would give, whatever order
// the GPU works in (the growth kernel in allocator.cu pops with atomics instead).
//
// The traffic is a few bytes per token and block (4.4 MB = 0.65 us at the measured copy rate
// for 4096 requests with 260,000 tokens), so launches and memory round trips bound it.  Up to
// BATCH_ONE_CTA requests and BATCH_FEW_TOKENS tokens it is one launch of one CTA.  More
// requests are scanned by one thread-block cluster, whose CTAs exchange their totals through
// distributed shared memory, with a cluster barrier where a launch would stand; more tokens
// are filled in by a second kernel over the whole GPU, launched early behind the first.
#include <cooperative_groups.h>

#include "pkv_common.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int BATCH_CTAS = 8;          // portable cluster size
constexpr int BATCH_THREADS = 1024;
// Requests of one CTA, one per thread: 100 requests 6.0 us (the cluster 9.2), 1000 with one token
// each 7.7 (10.5).
constexpr int BATCH_ONE_CTA = 1024;
// Tokens up to which the first kernel fills them in itself, one round of one CTA: 300 requests with
// 3400 tokens 7.8 us (8.6 with the second kernel), 2 with 5600 7.5 (6.4 with it), 1000 with 15000
// 17.2 (10.0 with it).
constexpr int BATCH_FEW_TOKENS = 4096;
constexpr int TOKENS_THREADS = 256;
constexpr int BATCH_WARPS = BATCH_THREADS / 32;

struct SeqNeed {
    int past, tokens, need, status;
};

// Lengths, blocks needed and the status that does not depend on the other requests.
__device__ __forceinline__ SeqNeed seq_need(const BatchParams& p, int s, bool report) {
    SeqNeed r;
    r.past = p.past_lens[s];
    const int nw = p.new_lens[s];
    r.tokens = nw > 0 ? nw : 0;
    r.need = 0;
    r.status = 0;
    // (no context reaches the last block of 2^31 positions: rounding up to blocks stays in range)
    const long long cap = min((long long)p.max_blocks_per_seq * p.block_size, 0x7fffffffll - p.block_size);
    if (r.past < 0 || nw < 0 || (long long)r.past + nw > cap) {
        r.status = 2;
        return r;
    }
    if (nw == 0) return r;
    const int held = (r.past + p.block_size - 1) / p.block_size;
    if (r.past % p.block_size != 0) {  // the last block held receives tokens: it must be this row's alone
        const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + held - 1];
        if ((unsigned)b >= (unsigned)p.alloc.num_blocks) {
            if (report) set_error(p.err, PKV_DEVERR_BLOCK_ID);
            r.status = 2;
            return r;
        }
        if (p.alloc.refcount[b] != 1) {
            r.status = 3;
            return r;
        }
    }
    r.need = (int)(((long long)r.past + nw + p.block_size - 1) / p.block_size) - held;
    return r;
}

struct Pair {
    long long tokens, need;
};

__device__ __forceinline__ Pair warp_inclusive(Pair v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(FULL_MASK, v.tokens, o);
        const long long b = __shfl_up_sync(FULL_MASK, v.need, o);
        if (lane >= o) {
            v.tokens += a;
            v.need += b;
        }
    }
    return v;
}

// Inclusive sums over the CTA's threads; `total` gets the CTA's sums.
__device__ __forceinline__ Pair block_inclusive(Pair v, Pair* warp_sums, Pair* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_inclusive(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = warp_inclusive(warp_sums[lane], lane);
    __syncthreads();
    if (warp > 0) {
        v.tokens += warp_sums[warp - 1].tokens;
        v.need += warp_sums[warp - 1].need;
    }
    *total = warp_sums[BATCH_WARPS - 1];
    __syncthreads();  // warp_sums is free again
    return v;
}

// The first of requests lo .. num_seqs - 1 that ends past token t (there is one).
__device__ __forceinline__ int request_of(const int* starts, int lo, int num_seqs, long long t) {
    int hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (starts[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// Four tokens in a row, the first of request s (when it is one of the `real` ones), with wide
// stores.  starts and ctxs are query_start and context_lens or copies of them.
__device__ __forceinline__ void fill_tokens(const BatchParams& p, long long t0, int real, int s, bool wide,
                                            const int* starts, const int* ctxs) {
    const int S = p.num_seqs, M = p.max_blocks_per_seq, B = p.block_size;
    int end = 0, next_pos = 0, ctx = 0;
    int pos[4], seq[4];
    long long slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long t = t0 + i;
        pos[i] = seq[i] = -1;
        slot[i] = -1;
        if (t >= real) continue;
        if (i == 0 || t >= end) {
            if (i > 0 && starts[++s + 1] <= t) s = request_of(starts, s + 1, S, t);
            end = starts[s + 1];
            ctx = ctxs[s];
            next_pos = ctx - (end - (int)t);
        }
        seq[i] = s;
        if (ctx > 0) {
            pos[i] = next_pos;
            const int id = p.block_tables[(size_t)s * M + next_pos / B];
            if (id >= 0) slot[i] = (long long)id * B + next_pos % B;
        }
        ++next_pos;
    }
    if (wide && t0 + 4 <= p.max_tokens) {
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(p.token_seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        longlong2* out = reinterpret_cast<longlong2*>(p.slot_mapping + t0);
        out[0] = make_longlong2(slot[0], slot[1]);
        out[1] = make_longlong2(slot[2], slot[3]);
    } else {
        for (int i = 0; i < 4 && t0 + i < p.max_tokens; ++i) {
            p.positions[t0 + i] = pos[i];
            p.token_seq[t0 + i] = seq[i];
            p.slot_mapping[t0 + i] = slot[i];
        }
    }
}

__device__ __forceinline__ bool wide_tokens(const BatchParams& p) {
    return ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.token_seq) |
             reinterpret_cast<uintptr_t>(p.slot_mapping)) & 15u) == 0;
}

}  // namespace

template <int CTAS>
__global__ void __launch_bounds__(BATCH_THREADS) build_batch_kernel(const BatchParams p, int fill) {
    static_assert(BATCH_WARPS == 32, "one lane per warp total");
    __shared__ Pair warp_sums[BATCH_WARPS];
    __shared__ Pair totals_s[CTAS];       // of every CTA, written by each into all
    __shared__ long long popped_s[CTAS];  // blocks popped up to each CTA's last served request: of rank 0
    __shared__ long long cta_popped;      // this CTA's
    __shared__ long long upto_s[BATCH_THREADS];  // inclusive block counts of the tile's requests
    __shared__ int first_s[BATCH_THREADS];       // first fresh logical block, -1: not served
    __shared__ int start_s[BATCH_THREADS + 1], ctx_s[BATCH_THREADS];  // one CTA: starts and contexts
    cg::cluster_group cluster = cg::this_cluster();
    // the token kernel may be set up meanwhile; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (CTAS > 1) cluster.barrier_arrive();  // running: its shared memory may be written to
    const int rank = CTAS > 1 ? (int)cluster.block_rank() : 0, tid = threadIdx.x;
    const int S = p.num_seqs, M = p.max_blocks_per_seq, B = p.block_size;
    const int per = (S + CTAS - 1) / CTAS;
    const int s_lo = min(S, rank * per), s_hi = min(S, s_lo + per);
    long long free_blocks = *p.alloc.free_count;
    free_blocks = free_blocks < 0 ? 0 : min(free_blocks, (long long)p.alloc.num_blocks);

    if (rank == 0 && tid == 0) p.query_start[0] = 0;

    // ---- this CTA's totals, then the sums of the CTAs before it
    SeqNeed held_need{0, 0, 0, 0};
    Pair base{0, 0};
    long long all_tokens = 0;
    if (tid == 0) cta_popped = 0;
    if (CTAS > 1) {
        Pair mine{0, 0}, total;
        for (int s = s_lo + tid; s < s_hi; s += BATCH_THREADS) {
            held_need = seq_need(p, s, true);
            mine.tokens += held_need.tokens;
            mine.need += held_need.need;
        }
        block_inclusive(mine, warp_sums, &total);
        cluster.barrier_wait();
        if (tid < CTAS) *cluster.map_shared_rank(&totals_s[rank], tid) = total;
        cluster.sync();  // also: every CTA has read the free count before it may be rewritten
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
            const Pair v = totals_s[r];
            all_tokens += v.tokens;
            if (r < rank) {
                base.tokens += v.tokens;
                base.need += v.need;
            }
        }
    } else {
        if (s_lo + tid < s_hi) held_need = seq_need(p, s_lo + tid, true);
        __syncthreads();
    }

    // ---- requests in tiles of one per thread: starts, contexts, statuses, table entries
    for (int s0 = s_lo; s0 < s_hi; s0 += BATCH_THREADS) {
        const int s = s0 + tid;
        const bool live = s < s_hi;
        // one tile per CTA in all but the largest batches: the first pass's values serve (their sums
        // within the CTA are made again)
        SeqNeed n{0, 0, 0, 0};
        if (live) n = (s_hi - s_lo <= BATCH_THREADS) ? held_need : seq_need(p, s, false);
        Pair tile;
        Pair v = block_inclusive(Pair{n.tokens, n.need}, warp_sums, &tile);
        v.tokens += base.tokens;
        v.need += base.need;
        if (live) {
            if (v.tokens > p.max_tokens && n.tokens > 0) n.status = 2;  // its rows are not in the batch
            if (n.status == 0 && n.need > 0 && v.need > free_blocks) n.status = 1;
            const int end = (int)min(v.tokens, (long long)p.max_tokens);
            const int ctx = n.status == 0 ? n.past + n.tokens : 0;
            p.query_start[s + 1] = end;
            p.context_lens[s] = ctx;
            if (CTAS == 1) {
                start_s[tid + 1] = end;
                ctx_s[tid] = ctx;
            }
            p.seq_status[s] = n.status;
            if (n.status == 0 && n.need > 0) atomicMax(&cta_popped, v.need);
        }
        upto_s[tid] = v.need;
        first_s[tid] = live && n.status == 0 ? (n.past + B - 1) / B : -1;
        __syncthreads();
        // the tile's fresh blocks, one per thread and step: the request is found by its count
        for (long long k = tid; k < tile.need; k += BATCH_THREADS) {
            const long long at = base.need + k;
            if (at >= free_blocks) break;  // past the stack: its request is not served
            const int id = p.alloc.free_ids[free_blocks - 1 - at];
            int lo = 0, hi = min(BATCH_THREADS, s_hi - s0) - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (upto_s[mid] > at) hi = mid; else lo = mid + 1;
            }
            if (first_s[lo] < 0) continue;
            const long long before = lo > 0 ? upto_s[lo - 1] : base.need;
            int32_t* entry = p.block_tables + (size_t)(s0 + lo) * M + first_s[lo] + (at - before);
            if ((unsigned)id >= (unsigned)p.alloc.num_blocks) {
                set_error(p.err, PKV_DEVERR_BLOCK_ID);  // not a free stack: no block is taken
                *entry = -1;
            } else {
                *entry = id;
                p.alloc.refcount[id] = 1;
            }
        }
        base.tokens += tile.tokens;
        base.need += tile.need;
        __syncthreads();
    }
    if (CTAS == 1) all_tokens = base.tokens;
    if (all_tokens > p.max_tokens && rank == 0 && tid == 0) set_error(p.err, PKV_DEVERR_POSITION);
    if (CTAS > 1) {
        if (tid == 0) *cluster.map_shared_rank(&popped_s[rank], 0) = cta_popped;
        cluster.sync();  // and starts, contexts and tables of every CTA are visible
    }
    if (rank == 0 && tid == 0) {
        long long popped = cta_popped;
#pragma unroll
        for (int r = 1; r < CTAS; ++r) popped = max(popped, popped_s[r]);
        *p.free_count_out = (int)(free_blocks - popped);
    }
    if (fill) {
        const int real = (int)min(all_tokens, (long long)p.max_tokens);
        const bool wide = wide_tokens(p);
        const int* starts = CTAS == 1 ? start_s : p.query_start;
        for (long long t0 = ((long long)rank * BATCH_THREADS + tid) * 4; t0 < p.max_tokens;
             t0 += (long long)CTAS * BATCH_THREADS * 4)
            fill_tokens(p, t0, real, t0 < real ? request_of(starts, 0, S, t0) : 0, wide, starts,
                        CTAS == 1 ? ctx_s : p.context_lens);
    }
}

__global__ void __launch_bounds__(TOKENS_THREADS) batch_tokens_kernel(const BatchParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int S = p.num_seqs, lane = threadIdx.x & 31;
    const int* starts = p.query_start;
    const long long t0 = ((long long)blockIdx.x * TOKENS_THREADS + threadIdx.x) * 4, w0 = t0 - 4 * lane;
    const int real = starts[S];
    int s = 0;
    if (w0 < real) {
        // the request of the warp's first token, 32 groups of requests at a time: two or three loads
        // behind one another where one lane's search would take twelve
        int lo = 0, n = S;
        while (n > 1) {
            const int step = (n + 31) / 32, first = lane * step;
            const bool past = first < n && starts[lo + min(first + step, n)] > w0;  // the group's last ends past it
            const int k = __ffs(__ballot_sync(FULL_MASK, past)) - 1;
            lo += k * step;
            n = min(step, n - k * step);
        }
        // that of each lane's: among the next 32, whose ends the lanes hold, or searched for
        const int end = starts[min(lo + lane, S - 1) + 1];
        int k = 0;
#pragma unroll
        for (int b = 16; b >= 1; b >>= 1)
            if (__shfl_sync(FULL_MASK, end, k + b - 1) <= t0) k += b;
        s = min(lo + k, S - 1);
        if (t0 < real && k == 31 && starts[s + 1] <= t0) s = request_of(starts, s, S, t0);
    }
    if (t0 < p.max_tokens) fill_tokens(p, t0, real, s, wide_tokens(p), starts, p.context_lens);
}

cudaError_t launch_build_batch(const BatchParams& p, cudaStream_t stream) {
    const bool one = p.num_seqs <= BATCH_ONE_CTA, fill = p.max_tokens <= BATCH_FEW_TOKENS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one ? 1 : BATCH_CTAS);
    cfg.blockDim = dim3(BATCH_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cfg.gridDim.x;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = one ? 0 : 1;
    cudaError_t e = one ? cudaLaunchKernelEx(&cfg, build_batch_kernel<1>, p, (int)fill)
                        : cudaLaunchKernelEx(&cfg, build_batch_kernel<BATCH_CTAS>, p, (int)fill);
    if (e != cudaSuccess || fill) return e;
    cfg.gridDim = dim3((unsigned)(((long long)p.max_tokens + 4 * TOKENS_THREADS - 1) / (4 * TOKENS_THREADS)));
    cfg.blockDim = dim3(TOKENS_THREADS);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, batch_tokens_kernel, p);
}

}  // namespace pkv
