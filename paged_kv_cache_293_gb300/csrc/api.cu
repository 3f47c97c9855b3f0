// api.cu -- the C ABI of libpagedkv.so (declared in include/pagedkv.h).
//
// Host-side argument checks, the choice of partition size, workspace layout,
// dispatch to the typed kernels, and the device error word.  Nothing here
// allocates device memory or synchronises, except pkv_get_device_error.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pkv_common.cuh"
#include "prefix.cuh"
#include "q8.cuh"

namespace {

// One word per device: kernels OR error bits into it instead of trapping.
__device__ unsigned int g_error_word;

constexpr int MAX_DEVICES = 64;
std::atomic<unsigned int*> g_error_ptr[MAX_DEVICES];  // looked up once per device

pkv_status error_word(unsigned int** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return PKV_ERR_CUDA;
    unsigned int* w = g_error_ptr[dev].load(std::memory_order_acquire);
    if (!w) {  // callers racing here all find the same address
        void* ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_error_word) != cudaSuccess) return PKV_ERR_CUDA;
        w = static_cast<unsigned int*>(ptr);
        g_error_ptr[dev].store(w, std::memory_order_release);
    }
    *out = w;
    return PKV_OK;
}

std::atomic<int> g_engine{PKV_ENGINE_AUTO};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pkv_status check_pool(const pkv_pool* pool) {
    if (!pool || !pool->k || !pool->v) return PKV_ERR_INVALID;
    if (!aligned16(pool->k) || !aligned16(pool->v)) return PKV_ERR_INVALID;
    if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->num_kv_heads <= 0 ||
        pool->head_dim <= 0)
        return PKV_ERR_INVALID;
    if (pool->dtype != PKV_F32 && pool->dtype != PKV_F16 && pool->dtype != PKV_BF16)
        return PKV_ERR_INVALID;
    if (pool->block_size != 16 && pool->block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (pool->head_dim != 64 && pool->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

int32_t ceil_div(int64_t a, int64_t b) { return int32_t((a + b - 1) / b); }

struct WsLayout {
    size_t l_off, o_off, bytes;
};

WsLayout ws_layout(int32_t S, int32_t Hq, int32_t D, int32_t parts) {
    const size_t rows = (size_t)S * Hq * parts;
    const size_t a = (rows * 4 + 15) & ~size_t(15);
    return WsLayout{a, 2 * a, 2 * a + rows * D * 4};
}

// One pass while the longest context is at most 3072 tokens; beyond that,
// 1024-token partitions (a multiple of 16 and 32), or 2048 with several query rows
// per sequence, whose partial results and merge cost num_queries times as much.
// Measured on the batches here: one pass was best for the LLaMA-7B (max 2048) and
// shared-prefix GQA (max 2560) batches, 1024-token partitions for LLaMA-13B (max
// 4096, a long lognormal tail) and the 32k-128k contexts; on the LLaMA-13B batch
// with 4 / 8 new tokens per sequence 2048-token partitions took 346.0 / 362.9 us
// against 348.6 / 371.8 us with 1024.
int32_t auto_partition(const pkv_pool* pool, int32_t max_context_len, int32_t num_queries = 1) {
    const int32_t B = pool->block_size;
    const int32_t one_pass_limit = 3072, split = num_queries > 1 ? 2048 : 1024;
    if (max_context_len <= one_pass_limit)
        return max_context_len <= 0 ? B : ceil_div(max_context_len, B) * B;
    return split;
}

struct DecodeArgs {
    const pkv_pool* pool;
    const void* q;
    int32_t S, Hq;
    const int32_t* bt;
    int32_t M;
    const int32_t* ctx;
    int32_t max_ctx;
    float scale;
    int32_t P;  // 0 = auto
    int32_t NQ = 1;  // query rows per sequence
};

pkv_status check_decode(const DecodeArgs& a) {
    pkv_status st = check_pool(a.pool);
    if (st != PKV_OK) return st;
    if (a.S < 0 || a.Hq <= 0 || a.M <= 0 || a.max_ctx < 0) return PKV_ERR_INVALID;
    if (a.Hq % a.pool->num_kv_heads != 0) return PKV_ERR_INVALID;
    if (!std::isfinite(a.scale)) return PKV_ERR_INVALID;
    if (a.P < 0 || (a.P > 0 && a.P % a.pool->block_size != 0)) return PKV_ERR_INVALID;
    if (a.S > 0 && (!a.q || !a.bt || !a.ctx)) return PKV_ERR_INVALID;
    if (a.S > 0 && !aligned16(a.q)) return PKV_ERR_INVALID;
    const int32_t G = a.Hq / a.pool->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
    if (a.S > 65535) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

cudaError_t launch_decode_typed(const pkv::DecodeParams& p, int32_t dtype, int D, int G,
                                cudaStream_t stream) {
    switch (dtype) {
        case PKV_F32: return pkv::launch_decode<float>(p, D, G, stream);
        case PKV_F16: return pkv::launch_decode<__half>(p, D, G, stream);
        default: return pkv::launch_decode<__nv_bfloat16>(p, D, G, stream);
    }
}

struct AppendArgs {
    const void* k_new;
    const void* v_new;
    int64_t* slot_out;
};

// Shared body of decode (direct = 1) and the partition step (direct = 0);
// `append` (may be null) turns on the fused write of each sequence's new token.
pkv_status run_decode(const DecodeArgs& a, void* out, int32_t out_dtype, int direct,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream,
                      const AppendArgs* append = nullptr) {
    const pkv_pool* pool = a.pool;
    const int32_t P = a.P > 0 ? a.P : auto_partition(pool, a.max_ctx, a.NQ);
    const int32_t parts = a.max_ctx > 0 ? ceil_div(a.max_ctx, P) : 1;
    if (parts > 65535) return PKV_ERR_UNSUPPORTED;
    const bool need_ws = !direct || parts > 1;
    const WsLayout lay = ws_layout(a.S * a.NQ, a.Hq, pool->head_dim, parts);
    if (need_ws && (!workspace || !aligned16(workspace) || workspace_bytes < lay.bytes))
        return PKV_ERR_WORKSPACE;
    if (a.S == 0) return PKV_OK;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;

    pkv::DecodeParams p{};
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.num_kv_heads = pool->num_kv_heads;
    p.q = a.q;
    p.num_seqs = a.S;
    p.num_q_heads = a.Hq;
    p.block_tables = a.bt;
    p.max_blocks_per_seq = a.M;
    p.context_lens = a.ctx;
    p.max_context_len = a.max_ctx;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.partition_size = P;
    p.max_parts = parts;
    p.out = out;
    p.out_dtype = out_dtype;
    p.direct_single = direct;
    const int G = a.Hq / pool->num_kv_heads;
    p.num_queries = a.NQ;
    p.queries_per_cta = 8 / G < a.NQ ? 8 / G : a.NQ;
    if (need_ws) {
        char* ws = static_cast<char*>(workspace);
        p.ws_m = reinterpret_cast<float*>(ws);
        p.ws_l = reinterpret_cast<float*>(ws + lay.l_off);
        p.ws_o = reinterpret_cast<float*>(ws + lay.o_off);
    }
    if (append) {
        p.k_new = append->k_new;
        p.v_new = append->v_new;
        p.slot_out = append->slot_out;
    }
    p.err = err;
    if (a.NQ > 1) {
        // several query rows per sequence: the tensor-core kernel only
        const cudaError_t e =
            pool->dtype == PKV_F16
                ? pkv::launch_decode_mma<__half>(p, pool->head_dim, G, stream)
                : pkv::launch_decode_mma<__nv_bfloat16>(p, pool->head_dim, G, stream);
        if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
        if (e != cudaSuccess) return PKV_ERR_CUDA;
    } else if (launch_decode_typed(p, pool->dtype, pool->head_dim, G, stream) != cudaSuccess) {
        return PKV_ERR_CUDA;
    }
    if (direct && parts > 1) {
        pkv::MergeParams mp{};
        mp.ws_m = p.ws_m;
        mp.ws_l = p.ws_l;
        mp.ws_o = p.ws_o;
        mp.context_lens = a.ctx;
        mp.num_seqs = a.S;
        mp.num_q_heads = a.Hq;
        mp.head_dim = pool->head_dim;
        mp.max_parts = parts;
        mp.partition_size = P;
        mp.skip_single = 1;
        mp.num_queries = a.NQ;
        mp.prefix_parts = 0;
        mp.skip_tokens = 0;
        mp.out = out;
        mp.out_dtype = out_dtype;
        mp.err = err;
        if (pkv::launch_merge(mp, stream) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace

bool pkv::use_tensor_cores(int group) {
    const int e = g_engine.load(std::memory_order_relaxed);
    return e == PKV_ENGINE_TENSOR_CORES || (e == PKV_ENGINE_AUTO && group >= 4);
}

// Partition scratch of pkv_paged_attention_decode_static_workspace, for callers
// that cannot allocate device memory: one fixed array per device, held for the
// life of the process, shared by every call of that entry point.
static __device__ __align__(256) unsigned char pkv_static_workspace[PKV_STATIC_WORKSPACE_BYTES];

namespace {

void* g_static_ws_ptr[MAX_DEVICES] = {nullptr};
cudaError_t g_static_ws_status[MAX_DEVICES];
std::once_flag g_static_ws_once[MAX_DEVICES];

// Device address of the array on the current device, looked up once per
// device with that device current.  Host code only sees a stand-in for the
// array's name, never a usable device address, so the kernels get this one.
pkv_status static_workspace(void** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return PKV_ERR_CUDA;
    std::call_once(g_static_ws_once[dev], [dev] {
        void* ptr = nullptr;
        g_static_ws_status[dev] = cudaGetSymbolAddress(&ptr, pkv_static_workspace);
        g_static_ws_ptr[dev] = ptr;
    });
    if (g_static_ws_status[dev] != cudaSuccess || !g_static_ws_ptr[dev]) return PKV_ERR_CUDA;
    *out = g_static_ws_ptr[dev];
    return PKV_OK;
}

}  // namespace

extern "C" {

int32_t pkv_version(void) { return 100; }

pkv_status pkv_set_decode_engine(int32_t engine) {
    if (engine != PKV_ENGINE_AUTO && engine != PKV_ENGINE_CUDA_CORES &&
        engine != PKV_ENGINE_TENSOR_CORES)
        return PKV_ERR_INVALID;
    g_engine.store(engine, std::memory_order_relaxed);
    return PKV_OK;
}

int32_t pkv_get_decode_engine(void) { return g_engine.load(std::memory_order_relaxed); }

const char* pkv_status_str(pkv_status status) {
    switch (status) {
        case PKV_OK: return "ok";
        case PKV_ERR_INVALID: return "invalid argument";
        case PKV_ERR_UNSUPPORTED: return "unsupported configuration";
        case PKV_ERR_WORKSPACE: return "workspace missing or too small";
        case PKV_ERR_CUDA: return "CUDA error";
        case PKV_ERR_DEVICE: return "device error flags set";
    }
    return "unknown status";
}

pkv_status pkv_slot_mapping(const int32_t* block_tables, int32_t max_blocks_per_seq,
                            int32_t num_seqs, const int32_t* positions, const int32_t* token_seq,
                            int32_t num_tokens, int32_t block_size, int64_t* slot_mapping,
                            void* stream) {
    if (num_tokens < 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_seqs < 0)
        return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!block_tables || !positions || !slot_mapping || num_seqs == 0) return PKV_ERR_INVALID;
    if (!token_seq && num_tokens > num_seqs) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_slot_mapping(block_tables, max_blocks_per_seq, num_seqs, positions,
                                    token_seq, num_tokens, block_size, slot_mapping, err,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_kv_cache_write(const pkv_pool* pool, const void* k_new, const void* v_new,
                              const int64_t* slot_mapping, int32_t num_tokens, void* stream) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !slot_mapping || !aligned16(k_new) || !aligned16(v_new))
        return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_cache_write(*pool, k_new, v_new, slot_mapping, num_tokens, err,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

int32_t pkv_choose_partition_size(const pkv_pool* pool, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t max_context_len) {
    (void)num_seqs;
    (void)num_q_heads;
    if (!pool || pool->block_size <= 0 || max_context_len < 0) return 0;
    return auto_partition(pool, max_context_len);
}

size_t pkv_decode_workspace_bytes(const pkv_pool* pool, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t max_context_len, int32_t partition_size) {
    if (!pool || pool->block_size <= 0 || pool->head_dim <= 0 || num_seqs < 0 ||
        num_q_heads <= 0 || max_context_len < 0 || partition_size < 0)
        return 0;
    const int32_t P = partition_size > 0 ? partition_size : auto_partition(pool, max_context_len);
    const int32_t parts = max_context_len > 0 ? ceil_div(max_context_len, P) : 1;
    if (parts <= 1) return 0;
    return ws_layout(num_seqs, num_q_heads, pool->head_dim, parts).bytes;
}

size_t pkv_partition_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                                     int32_t max_context_len, int32_t partition_size) {
    if (num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || max_context_len < 0 ||
        partition_size <= 0)
        return 0;
    const int32_t parts = max_context_len > 0 ? ceil_div(max_context_len, partition_size) : 1;
    return ws_layout(num_seqs, num_q_heads, head_dim, parts).bytes;
}

pkv_status pkv_paged_attention_decode(const pkv_pool* pool, const void* q, int32_t num_seqs,
                                      int32_t num_q_heads, const int32_t* block_tables,
                                      int32_t max_blocks_per_seq, const int32_t* context_lens,
                                      int32_t max_context_len, float scale, void* out,
                                      int32_t out_dtype, int32_t partition_size, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (num_seqs > 0 && !out) return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    return run_decode(a, out, out_dtype, 1, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream));
}

pkv_status pkv_paged_attention_decode_static_workspace(
    const pkv_pool* pool, const void* q, int32_t num_seqs, int32_t num_q_heads,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t max_context_len, float scale, void* out, int32_t out_dtype, int32_t partition_size,
    void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (num_seqs > 0 && !out) return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    const size_t need = pkv_decode_workspace_bytes(pool, num_seqs, num_q_heads, max_context_len,
                                                   partition_size);
    if (need > PKV_STATIC_WORKSPACE_BYTES) return PKV_ERR_WORKSPACE;
    if (num_seqs == 0) return PKV_OK;
    void* ws = nullptr;
    st = static_workspace(&ws);
    if (st != PKV_OK) return st;
    return run_decode(a, out, out_dtype, 1, ws, PKV_STATIC_WORKSPACE_BYTES,
                      static_cast<cudaStream_t>(stream));
}

pkv_status pkv_paged_attention_decode_append(
    const pkv_pool* pool, const void* q, const void* k_new, const void* v_new, int32_t num_seqs,
    int32_t num_q_heads, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, int32_t max_context_len, float scale, void* out,
    int32_t out_dtype, int32_t partition_size, void* workspace, size_t workspace_bytes,
    int64_t* slot_mapping, void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (num_seqs > 0 && (!out || !k_new || !v_new)) return PKV_ERR_INVALID;
    if (num_seqs > 0 && (!aligned16(k_new) || !aligned16(v_new))) return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    const AppendArgs app{k_new, v_new, slot_mapping};
    return run_decode(a, out, out_dtype, 1, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream), &app);
}

pkv_status pkv_paged_attention_decode_multi(
    const pkv_pool* pool, const void* q, int32_t num_queries, int32_t num_seqs,
    int32_t num_q_heads, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, int32_t max_context_len, float scale, void* out,
    int32_t out_dtype, int32_t partition_size, void* workspace, size_t workspace_bytes,
    void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (num_queries < 1 || (int64_t)num_seqs * num_queries > INT32_MAX) return PKV_ERR_INVALID;
    if (num_seqs > 0 && !out) return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    if (pool->dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
    a.NQ = num_queries;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    if ((int64_t)pool->num_kv_heads * ((num_queries + 8 / G - 1) / (8 / G)) > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    return run_decode(a, out, out_dtype, 1, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream));
}

pkv_status pkv_paged_attention_decode_multi_append(
    const pkv_pool* pool, const void* q, const void* k_new, const void* v_new,
    int32_t num_queries, int32_t num_seqs, int32_t num_q_heads, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len,
    float scale, void* out, int32_t out_dtype, int32_t partition_size, void* workspace,
    size_t workspace_bytes, int64_t* slot_mapping, void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)))
        return PKV_ERR_INVALID;
    if (num_queries == 1)
        return pkv_paged_attention_decode_append(pool, q, k_new, v_new, num_seqs, num_q_heads,
                                                 block_tables, max_blocks_per_seq, context_lens,
                                                 max_context_len, scale, out, out_dtype,
                                                 partition_size, workspace, workspace_bytes,
                                                 slot_mapping, stream);
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (num_queries < 1 || (int64_t)num_seqs * num_queries > INT32_MAX) return PKV_ERR_INVALID;
    if (num_seqs > 0 && !out) return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    if (pool->dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
    a.NQ = num_queries;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    if ((int64_t)pool->num_kv_heads * ((num_queries + 8 / G - 1) / (8 / G)) > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    const AppendArgs app{k_new, v_new, slot_mapping};
    return run_decode(a, out, out_dtype, 1, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream), &app);
}

namespace {

struct CascadeShape {
    int32_t P, suffix_parts, prefix_splits, tokens_per_split, max_parts;
};

// Streaming multiprocessors of the current device (152 when it cannot be asked).
int32_t sm_count() {
    static std::atomic<int32_t> cached[64];  // 0 until asked; racing callers agree
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int32_t n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 152;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// The prefix pass runs two CTAs per SM over (kv head, 128-row tile, split of the
// prefix); the split count minimises waves x (64-token chunks per split + 3), the 3
// standing for a CTA's fixed cost (query tile, pipeline fill, epilogue).  Each split
// writes one slot, followed by the suffix partitions.
CascadeShape cascade_shape(const pkv_pool* pool, int32_t num_seqs, int32_t num_q_heads,
                           int32_t max_ctx, int32_t prefix_len, int32_t partition_size) {
    const int32_t rest = max_ctx > prefix_len ? max_ctx - prefix_len : 0;
    const int32_t P = partition_size > 0 ? partition_size : auto_partition(pool, rest);
    const int32_t sp = rest > 0 ? ceil_div(rest, P) : 1;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    const int64_t ctas = std::max<int64_t>(
        1, (int64_t)pool->num_kv_heads * (((int64_t)num_seqs * G + 127) / 128));
    const int64_t sms = sm_count();
    const int32_t chunks = std::max<int32_t>(1, ceil_div(prefix_len, 64));
    int32_t best_cps = chunks;
    int64_t best_cost = INT64_MAX;
    for (int32_t s = 1; s <= std::min<int32_t>(chunks, 64); ++s) {
        const int32_t cps = ceil_div(chunks, s);
        const int64_t splits = ceil_div(chunks, cps);
        const int64_t waves = (ctas * splits + 2 * sms - 1) / (2 * sms);  // two CTAs per SM
        const int64_t cost = waves * (cps + 3);
        if (cost < best_cost) {
            best_cost = cost;
            best_cps = cps;
        }
    }
    const int32_t splits = ceil_div(chunks, best_cps);
    return CascadeShape{P, sp, splits, best_cps * 64, splits + sp};
}

}  // namespace

size_t pkv_cascade_workspace_bytes(const pkv_pool* pool, int32_t num_seqs, int32_t num_q_heads,
                                   int32_t max_context_len, int32_t prefix_len,
                                   int32_t partition_size) {
    if (!pool || pool->block_size <= 0 || pool->head_dim <= 0 || num_seqs < 0 ||
        num_q_heads <= 0 || max_context_len < 0 || prefix_len <= 0 || partition_size < 0)
        return 0;
    if (num_q_heads % pool->num_kv_heads != 0) return 0;
    const CascadeShape c =
        cascade_shape(pool, num_seqs, num_q_heads, max_context_len, prefix_len, partition_size);
    return ws_layout(num_seqs, num_q_heads, pool->head_dim, c.max_parts).bytes;
}

pkv_status pkv_paged_attention_decode_cascade(
    const pkv_pool* pool, const void* q, int32_t num_seqs, int32_t num_q_heads,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t max_context_len, float scale, int32_t prefix_len, void* out, int32_t out_dtype,
    int32_t partition_size, const void* k_new, const void* v_new, int64_t* slot_mapping,
    void* workspace, size_t workspace_bytes, void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (pool->dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != PKV_F32 && out_dtype != pool->dtype) return PKV_ERR_UNSUPPORTED;
    if (prefix_len <= 0 || prefix_len % 16 != 0 || prefix_len % pool->block_size != 0 ||
        prefix_len > max_context_len || (int64_t)prefix_len > (int64_t)max_blocks_per_seq * pool->block_size)
        return PKV_ERR_INVALID;
    if ((k_new == nullptr) != (v_new == nullptr)) return PKV_ERR_INVALID;
    if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return PKV_ERR_INVALID;
    if (num_seqs > 0 && !out) return PKV_ERR_INVALID;
    const CascadeShape c =
        cascade_shape(pool, num_seqs, num_q_heads, max_context_len, prefix_len, partition_size);
    if (c.suffix_parts > 65535) return PKV_ERR_UNSUPPORTED;
    const WsLayout lay = ws_layout(num_seqs, num_q_heads, pool->head_dim, c.max_parts);
    if (!workspace || !aligned16(workspace) || workspace_bytes < lay.bytes) return PKV_ERR_WORKSPACE;
    // the prefix pass's limits (tensor-map rows, 128-row tiles in grid.y), checked before
    // anything is launched
    if ((int64_t)pool->num_blocks * pool->num_kv_heads * pool->block_size >= (1ll << 31) ||
        ((int64_t)num_seqs * (num_q_heads / pool->num_kv_heads) + 127) / 128 > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    unsigned int* err = nullptr;
    st = error_word(&err);
    if (st != PKV_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    float* ws_m = reinterpret_cast<float*>(ws);
    float* ws_l = reinterpret_cast<float*>(ws + lay.l_off);
    float* ws_o = reinterpret_cast<float*>(ws + lay.o_off);
    const int G = num_q_heads / pool->num_kv_heads;

    pkv::DecodeParams p{};
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.num_kv_heads = pool->num_kv_heads;
    p.q = q;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.partition_size = c.P;
    p.max_parts = c.max_parts;
    p.out = out;
    p.out_dtype = out_dtype;
    p.direct_single = 0;
    p.skip_tokens = prefix_len;
    p.part_offset = c.prefix_splits;
    p.num_queries = 1;
    p.queries_per_cta = 1;
    p.ws_m = ws_m;
    p.ws_l = ws_l;
    p.ws_o = ws_o;
    p.k_new = k_new;
    p.v_new = v_new;
    p.slot_out = slot_mapping;
    p.err = err;
    // the suffix decode's grid covers max_parts - part_offset = suffix partitions.  It goes
    // first and lets the prefix pass start on the SMs its last CTAs leave idle (the two
    // read and write disjoint data); the prefix pass ends only after it.
    p.trigger_dependents = 1;
    if (launch_decode_typed(p, pool->dtype, pool->head_dim, G, s) != cudaSuccess)
        return PKV_ERR_CUDA;

    pkv::PrefixParams pp{};
    pp.q = q;
    pp.num_seqs = num_seqs;
    pp.num_q_heads = num_q_heads;
    pp.num_kv_heads = pool->num_kv_heads;
    pp.num_blocks = pool->num_blocks;
    pp.block_size = pool->block_size;
    pp.block_tables = block_tables;
    pp.max_blocks_per_seq = max_blocks_per_seq;
    pp.prefix_len = prefix_len;
    pp.scale_log2 = scale * 1.4426950408889634f;
    pp.max_parts = c.max_parts;
    pp.tokens_per_split = c.tokens_per_split;
    pp.ws_m = ws_m;
    pp.ws_l = ws_l;
    pp.ws_o = ws_o;
    pp.err = err;
    cudaError_t e = pool->dtype == PKV_F16
                        ? pkv::launch_prefix<__half>(pp, pool->k, pool->v, pool->head_dim, s)
                        : pkv::launch_prefix<__nv_bfloat16>(pp, pool->k, pool->v, pool->head_dim, s);
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return PKV_ERR_CUDA;

    pkv::MergeParams mp{};
    mp.ws_m = ws_m;
    mp.ws_l = ws_l;
    mp.ws_o = ws_o;
    mp.context_lens = context_lens;
    mp.num_seqs = num_seqs;
    mp.num_q_heads = num_q_heads;
    mp.head_dim = pool->head_dim;
    mp.max_parts = c.max_parts;
    mp.partition_size = c.P;
    mp.skip_single = 0;
    mp.num_queries = 1;
    mp.prefix_parts = c.prefix_splits;
    mp.skip_tokens = prefix_len;
    mp.out = out;
    mp.out_dtype = out_dtype;
    mp.err = err;
    return pkv::launch_merge(mp, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_paged_attention_partitions(const pkv_pool* pool, const void* q, int32_t num_seqs,
                                          int32_t num_q_heads, const int32_t* block_tables,
                                          int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, int32_t max_context_len,
                                          float scale, int32_t partition_size, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    DecodeArgs a{pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq,
                 context_lens, max_context_len, scale, partition_size};
    pkv_status st = check_decode(a);
    if (st != PKV_OK) return st;
    if (partition_size <= 0) return PKV_ERR_INVALID;
    return run_decode(a, nullptr, PKV_F32, 0, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream));
}

pkv_status pkv_lse_merge(const void* workspace, size_t workspace_bytes, int32_t num_seqs,
                         int32_t num_q_heads, int32_t head_dim, const int32_t* context_lens,
                         int32_t max_context_len, int32_t partition_size, void* out,
                         int32_t out_dtype, void* stream) {
    if (num_seqs < 0 || num_q_heads <= 0 || max_context_len < 0 || partition_size <= 0)
        return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
        return PKV_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!context_lens || !out) return PKV_ERR_INVALID;
    const int32_t parts = max_context_len > 0 ? ceil_div(max_context_len, partition_size) : 1;
    const WsLayout lay = ws_layout(num_seqs, num_q_heads, head_dim, parts);
    if (!workspace || !aligned16(workspace) || workspace_bytes < lay.bytes) return PKV_ERR_WORKSPACE;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    const char* ws = static_cast<const char*>(workspace);
    pkv::MergeParams mp{};
    mp.ws_m = reinterpret_cast<const float*>(ws);
    mp.ws_l = reinterpret_cast<const float*>(ws + lay.l_off);
    mp.ws_o = reinterpret_cast<const float*>(ws + lay.o_off);
    mp.context_lens = context_lens;
    mp.num_seqs = num_seqs;
    mp.num_q_heads = num_q_heads;
    mp.head_dim = head_dim;
    mp.max_parts = parts;
    mp.partition_size = partition_size;
    mp.skip_single = 0;
    mp.num_queries = 1;
    mp.prefix_parts = 0;
    mp.skip_tokens = 0;
    mp.out = out;
    mp.out_dtype = out_dtype;
    mp.err = err;
    return pkv::launch_merge(mp, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                 : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks(const pkv_pool* pool, const int32_t* src_dst_pairs, int32_t num_pairs,
                           void* stream) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!src_dst_pairs) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_copy_blocks(*pool, *pool, src_dst_pairs, num_pairs, err,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

namespace {

// Device address of a pointer the kernels will dereference: device and managed
// memory as they are, pinned host memory through its mapped device address.
// Pageable host memory the runtime does not know is refused rather than risked.
bool device_addressable(const void* p, const void** out) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    switch (attr.type) {
        case cudaMemoryTypeDevice:
        case cudaMemoryTypeManaged:
            *out = p;
            return true;
        case cudaMemoryTypeHost:
            *out = attr.devicePointer;
            return attr.devicePointer != nullptr;
        default:
            return false;
    }
}

}  // namespace

pkv_status pkv_swap_blocks(const pkv_pool* src, const pkv_pool* dst, const int32_t* src_dst_pairs,
                           int32_t num_pairs, void* stream) {
    pkv_status st = check_pool(src);
    if (st != PKV_OK) return st;
    st = check_pool(dst);
    if (st != PKV_OK) return st;
    if (src->dtype != dst->dtype || src->block_size != dst->block_size ||
        src->num_kv_heads != dst->num_kv_heads || src->head_dim != dst->head_dim)
        return PKV_ERR_INVALID;
    if (num_pairs < 0) return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!src_dst_pairs) return PKV_ERR_INVALID;
    pkv_pool s2 = *src, d2 = *dst;
    const void* pairs = nullptr;
    const void *sk, *sv, *dk, *dv;
    if (!device_addressable(src->k, &sk) || !device_addressable(src->v, &sv) ||
        !device_addressable(dst->k, &dk) || !device_addressable(dst->v, &dv) ||
        !device_addressable(src_dst_pairs, &pairs))
        return PKV_ERR_INVALID;
    s2.k = const_cast<void*>(sk);
    s2.v = const_cast<void*>(sv);
    d2.k = const_cast<void*>(dk);
    d2.v = const_cast<void*>(dv);
    unsigned int* err = nullptr;
    st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_copy_blocks(s2, d2, static_cast<const int32_t*>(pairs), num_pairs, err,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

static bool allocator_ok(const pkv_block_allocator* a) {
    return a && a->free_ids && a->free_count && a->refcount && a->num_blocks > 0;
}

static pkv::AllocatorState allocator_state(const pkv_block_allocator* a) {
    return pkv::AllocatorState{a->free_ids, a->free_count, a->refcount, a->num_blocks};
}

pkv_status pkv_allocator_reset(const pkv_block_allocator* alloc, void* stream) {
    if (!allocator_ok(alloc)) return PKV_ERR_INVALID;
    return pkv::launch_allocator_reset(allocator_state(alloc), static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_allocate_for_append(const pkv_block_allocator* alloc, const pkv_pool* pool,
                                   int32_t* block_tables, int32_t max_blocks_per_seq,
                                   const int32_t* old_lens, const int32_t* new_lens,
                                   int32_t num_seqs, int32_t* seq_status, void* stream) {
    if (!allocator_ok(alloc)) return PKV_ERR_INVALID;
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (alloc->num_blocks != pool->num_blocks || max_blocks_per_seq <= 0 || num_seqs < 0)
        return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !old_lens || !new_lens || !seq_status) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_allocate_for_append(allocator_state(alloc), *pool, block_tables,
                                           max_blocks_per_seq, old_lens, new_lens, num_seqs,
                                           seq_status, err, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_fork_sequences(const pkv_block_allocator* alloc, int32_t block_size,
                              int32_t* block_tables, int32_t max_blocks_per_seq,
                              const int32_t* src_dst_seqs, const int32_t* lens,
                              int32_t num_pairs, void* stream) {
    if (!allocator_ok(alloc) || block_size <= 0 || max_blocks_per_seq <= 0 || num_pairs < 0)
        return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!block_tables || !src_dst_seqs || !lens) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_fork_sequences(allocator_state(alloc), block_size, block_tables,
                                      max_blocks_per_seq, src_dst_seqs, lens, num_pairs, err,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_free_sequences(const pkv_block_allocator* alloc, int32_t block_size,
                              int32_t* block_tables, int32_t max_blocks_per_seq,
                              const int32_t* seqs, const int32_t* lens, int32_t num_seqs,
                              void* stream) {
    if (!allocator_ok(alloc) || block_size <= 0 || max_blocks_per_seq <= 0 || num_seqs < 0)
        return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !seqs || !lens) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    return pkv::launch_free_sequences(allocator_state(alloc), block_size, block_tables,
                                      max_blocks_per_seq, seqs, lens, num_seqs, err,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_build_batch(const pkv_block_allocator* alloc, int32_t block_size,
                           int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* past_lens, const int32_t* new_lens, int32_t num_seqs,
                           int32_t max_tokens, int32_t* free_count_out, int32_t* query_start,
                           int32_t* context_lens, int32_t* positions, int32_t* token_seq,
                           int64_t* slot_mapping, int32_t* seq_status, void* stream) {
    if (!allocator_ok(alloc) || block_size <= 0 || max_blocks_per_seq <= 0 || num_seqs < 0 ||
        max_tokens < 0)
        return PKV_ERR_INVALID;
    if (!query_start) return PKV_ERR_INVALID;
    if (num_seqs > 0 && (!block_tables || !past_lens || !new_lens || !context_lens || !seq_status))
        return PKV_ERR_INVALID;
    if (max_tokens > 0 && (!positions || !token_seq || !slot_mapping)) return PKV_ERR_INVALID;
    pkv::BatchParams p{};
    pkv_status st = error_word(&p.err);
    if (st != PKV_OK) return st;
    p.alloc = allocator_state(alloc);
    p.block_size = block_size;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.past_lens = past_lens;
    p.new_lens = new_lens;
    p.num_seqs = num_seqs;
    p.max_tokens = max_tokens;
    p.free_count_out = free_count_out ? free_count_out : alloc->free_count;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.positions = positions;
    p.token_seq = token_seq;
    p.slot_mapping = slot_mapping;
    p.seq_status = seq_status;
    return pkv::launch_build_batch(p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

namespace {

// Whether any of n rows of `width` bytes, `stride` >= width apart from a on, shares a byte with
// the `bytes` from b on.
bool rows_overlap(const void* a, int64_t stride, int64_t width, int64_t n, const void* b, int64_t bytes) {
    if (!a || !b || n <= 0 || width <= 0 || bytes <= 0) return false;
    if (n == 1) stride = width;
    // the first row that ends past b
    const int64_t to_b = static_cast<const char*>(b) - static_cast<const char*>(a);
    const int64_t t = to_b < width ? 0 : (to_b - width) / stride + 1;
    return t < n && t * stride < to_b + bytes;
}

}  // namespace

namespace {

// The arguments that both writes of turned rows take, checked and as their kernels want them; the
// pools are checked before, `size` is an element of q's, k's and v's, `cache_bytes` those of a pool.
pkv_status rope_params(pkv::RopeParams& p, int64_t size, void* k_pool, void* v_pool, int64_t cache_bytes,
                       const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int32_t num_tokens, int32_t num_q_heads, const void* q_weight,
                       const void* k_weight, float eps, const float* cos_sin, int32_t max_position,
                       int32_t rotary_dim, int32_t interleaved, const int32_t* positions,
                       const int64_t* slot_mapping, void* q_out) {
    if (num_tokens < 0 || num_q_heads <= 0 || rotary_dim < 0 || rotary_dim > p.head_dim)
        return PKV_ERR_INVALID;
    if (!std::isfinite(eps) || eps < 0.f) return PKV_ERR_INVALID;
    if ((rotary_dim > 0) != (cos_sin != nullptr) || (rotary_dim > 0 && max_position <= 0))
        return PKV_ERR_INVALID;
    if (rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (num_q_heads > INT32_MAX - 2 * (int64_t)p.num_kv_heads) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !v || !q_out || !positions || !slot_mapping) return PKV_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin))
        return PKV_ERR_INVALID;
    // a row of heads is packed; rows may be further apart, by whole 16-byte vectors
    const int64_t vec = 16 / size, D = p.head_dim;
    const int64_t need_q = num_q_heads * D, need_kv = p.num_kv_heads * D;
    if (q_stride % vec != 0 || k_stride % vec != 0 || v_stride % vec != 0) return PKV_ERR_INVALID;
    if (num_tokens > 1 && (q_stride < need_q || k_stride < need_kv || v_stride < need_kv))
        return PKV_ERR_INVALID;
    // q_out may be q, row for row; otherwise tokens are read after others have been written
    const int64_t T = num_tokens, out_bytes = T * need_q * size;
    auto apart = [&](const void* in, int64_t bytes) { return !rows_overlap(in, bytes, bytes, 1, q_out, out_bytes); };
    const bool in_place = q_out == q && (T == 1 || q_stride == need_q);
    if ((!in_place && rows_overlap(q, q_stride * size, need_q * size, T, q_out, out_bytes)) ||
        rows_overlap(k, k_stride * size, need_kv * size, T, q_out, out_bytes) ||
        rows_overlap(v, v_stride * size, need_kv * size, T, q_out, out_bytes) ||
        !apart(k_pool, cache_bytes) || !apart(v_pool, cache_bytes) || !apart(q_weight, D * size) ||
        !apart(k_weight, D * size) || !apart(cos_sin, (int64_t)max_position * rotary_dim * 4) ||
        !apart(positions, T * 4) || !apart(slot_mapping, T * 8))
        return PKV_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.q_out = q_out;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    return PKV_OK;
}

}  // namespace

pkv_status pkv_qk_norm_rope_write(const pkv_pool* pool, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                  int32_t num_tokens, int32_t num_q_heads, const void* q_weight,
                                  const void* k_weight, float eps, const float* cos_sin,
                                  int32_t max_position, int32_t rotary_dim, int32_t interleaved,
                                  const int32_t* positions, const int64_t* slot_mapping,
                                  void* q_out, void* stream) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    const int64_t size = pool->dtype == PKV_F32 ? 4 : 2;
    pkv::RopeParams p{};
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.num_kv_heads = pool->num_kv_heads;
    p.head_dim = pool->head_dim;
    st = rope_params(p, size, pool->k, pool->v,
                     (int64_t)pool->num_blocks * pool->block_size * pool->num_kv_heads * pool->head_dim * size, q,
                     q_stride, k, k_stride, v, v_stride, num_tokens, num_q_heads, q_weight, k_weight, eps, cos_sin,
                     max_position, rotary_dim, interleaved, positions, slot_mapping, q_out);
    if (st != PKV_OK || num_tokens == 0) return st;
    st = error_word(&p.err);
    if (st != PKV_OK) return st;
    return pkv::launch_rope_write(p, pool->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

namespace {

// Sizes of a chunk attention call and where its workspace's parts lie.
struct ChunkShape {
    int64_t tiles, pieces, cut_pieces, partial_rows;
    size_t tile_start, tile, piece, merge, m, l, o, totals, bytes;
};

ChunkShape chunk_shape(int64_t Hkv, int32_t D, int32_t T, int32_t S, int32_t Hq, int32_t max_ctx) {
    const int64_t G = Hq / Hkv, sms = sm_count();
    const int64_t QT = 2 * (128 / G);  // queries per tile
    ChunkShape c{};
    c.tiles = std::min<int64_t>(T, T / QT + S);
    const int64_t steps = (max_ctx + (int64_t)pkv::CHUNK_TILE - 1) / pkv::CHUNK_TILE;
    const bool cuts = steps >= pkv::CHUNK_SPLIT_MIN;
    c.cut_pieces = cuts ? std::min<int64_t>(8 * sms, c.tiles * Hkv * 32) : 0;
    c.partial_rows = cuts ? std::min<int64_t>(3 * sms * 256, (int64_t)T * Hq * 32) : 0;
    c.pieces = c.tiles * Hkv + c.cut_pieces;
    size_t at = 128;  // header
    auto take = [&at](size_t bytes) {
        const size_t here = at;
        at = (at + bytes + 127) & ~size_t(127);
        return here;
    };
    c.tile_start = take(((size_t)S + 1) * 4);
    c.tile = take((size_t)c.tiles * sizeof(int4));
    c.piece = take((size_t)c.pieces * sizeof(pkv::ChunkPiece));
    c.merge = take((size_t)(c.cut_pieces / 2) * sizeof(pkv::ChunkMerge));
    c.m = take((size_t)c.partial_rows * 4);
    c.l = take((size_t)c.partial_rows * 4);
    c.o = take((size_t)c.partial_rows * D * 4);
    // two tiles of 128 rows per CTA
    const int64_t totals = std::min(c.pieces, sms) * 256 * (D + 4);
    c.totals = take(steps > pkv::CHUNK_SUM_STEPS ? (size_t)totals * 4 : 0);
    c.bytes = at;
    return c;
}

}  // namespace

namespace {

// The pool of a chunk attention call: 16-bit, or 8-bit with its scales.
struct ChunkPool {
    const void *k, *v;
    const float *k_scale, *v_scale;  // null: 16-bit
    int32_t num_blocks, block_size, num_kv_heads, head_dim, dtype;
};

size_t chunk_workspace(const ChunkPool& pool, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                       int32_t max_context_len) {
    if (pool.num_kv_heads <= 0 || pool.head_dim <= 0 || num_tokens < 0 || num_seqs < 0 ||
        num_q_heads <= 0 || max_context_len < 0 || num_q_heads % pool.num_kv_heads != 0 ||
        num_q_heads / pool.num_kv_heads > 128)
        return 0;
    return chunk_shape(pool.num_kv_heads, pool.head_dim, num_tokens, num_seqs, num_q_heads, max_context_len).bytes;
}

pkv_status run_chunk(const ChunkPool& pool, const void* q, int32_t num_tokens, int32_t num_q_heads,
                     const int32_t* query_start, int32_t num_seqs, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len, float scale,
                     void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 ||
        max_context_len < 0 || num_q_heads % pool.num_kv_heads != 0 || !std::isfinite(scale))
        return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != pool.dtype) return PKV_ERR_UNSUPPORTED;
    const int32_t G = num_q_heads / pool.num_kv_heads;
    if (pool.dtype == PKV_F32 || G > 128) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)pool.num_blocks * pool.num_kv_heads * pool.block_size >= (1ll << 31))
        return PKV_ERR_UNSUPPORTED;  // tensor-copy rows are int32
    // one CTA may have a whole context, and the kernel's waits end after about 2 s
    if (std::min<int64_t>((int64_t)max_blocks_per_seq * pool.block_size, max_context_len) > pkv::CHUNK_MAX_CONTEXT)
        return PKV_ERR_UNSUPPORTED;
    const ChunkShape c =
        chunk_shape(pool.num_kv_heads, pool.head_dim, num_tokens, num_seqs, num_q_heads, max_context_len);
    if (c.pieces > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0 || num_seqs == 0) return PKV_OK;
    if (!q || !query_start || !block_tables || !context_lens || !out || !aligned16(q) || !aligned16(out))
        return PKV_ERR_INVALID;
    if (!workspace || !aligned16(workspace) || workspace_bytes < c.bytes) return PKV_ERR_WORKSPACE;
    unsigned int* err = nullptr;
    const pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const int32_t sms = sm_count();

    pkv::ChunkTensors x{q, pool.k, pool.v, num_tokens, (int32_t)std::min<int64_t>(c.pieces, sms), c.tiles};
    pkv::ChunkPlanParams pl{};
    pl.query_start = query_start;
    pl.context_lens = context_lens;
    pl.num_seqs = num_seqs;
    pl.num_tokens = num_tokens;
    pl.max_blocks_per_seq = max_blocks_per_seq;
    pl.block_size = pool.block_size;
    pl.max_context_len = max_context_len;
    pl.num_kv_heads = pool.num_kv_heads;
    pl.group = G;
    pl.num_sms = sms;
    pl.ctas = x.ctas;
    pl.max_partial_rows = c.partial_rows;
    pl.max_cut_pieces = c.cut_pieces;
    pl.header = reinterpret_cast<int32_t*>(ws);
    pl.tile_start = reinterpret_cast<int32_t*>(ws + c.tile_start);
    pl.tiles = reinterpret_cast<int4*>(ws + c.tile);
    pl.pieces = reinterpret_cast<pkv::ChunkPiece*>(ws + c.piece);
    pl.merges = reinterpret_cast<pkv::ChunkMerge*>(ws + c.merge);
    pl.err = err;

    pkv::ChunkParams p{};
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = pool.num_kv_heads;
    p.group = G;
    p.head_dim = pool.head_dim;
    p.num_blocks = pool.num_blocks;
    p.block_size = pool.block_size;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    // the kernel takes maxima before scaling, which a positive scale allows: a negative one
    // negates the product instead, and a zero one becomes so small that every weight is 1
    const float size = std::fabs(scale) * 1.4426950408889634f;
    p.scale_log2 = size > 0.f ? size : 1e-30f;
    p.negate = scale < 0.f;
    p.out = out;
    p.out_dtype = out_dtype;
    p.header = pl.header;
    p.pieces = pl.pieces;
    p.merges = pl.merges;
    p.part_m = reinterpret_cast<float*>(ws + c.m);
    p.part_l = reinterpret_cast<float*>(ws + c.l);
    p.part_o = reinterpret_cast<float*>(ws + c.o);
    p.totals = reinterpret_cast<float*>(ws + c.totals);
    p.k_scale = pool.k_scale;
    p.v_scale = pool.v_scale;
    p.err = err;
    const bool f16 = pool.dtype == PKV_F16;
    const cudaError_t e = pool.k_scale ? (f16 ? pkv::launch_chunk_q8<__half>(pl, p, x, s)
                                              : pkv::launch_chunk_q8<__nv_bfloat16>(pl, p, x, s))
                                       : (f16 ? pkv::launch_chunk<__half>(pl, p, x, s)
                                              : pkv::launch_chunk<__nv_bfloat16>(pl, p, x, s));
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    if (c.partial_rows == 0) return PKV_OK;
    // half of what the GPU holds at a time: few to set up where nothing was cut (24 requests of up to
    // 512 queries 30.6 -> 29.8 us against 16 per SM; with 1 per SM 500 tokens over 130,500 take 735
    // us and not 700)
    const int64_t merge_ctas = std::min<int64_t>(
        4 * (int64_t)sms, std::max(c.tiles * pool.num_kv_heads, ((int64_t)num_tokens * num_q_heads + 7) / 8));
    return pkv::launch_chunk_merge(p, (int)merge_ctas, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

ChunkPool chunk_pool(const pkv_pool* p) {
    return {p->k, p->v, nullptr, nullptr, p->num_blocks, p->block_size, p->num_kv_heads, p->head_dim, p->dtype};
}

ChunkPool chunk_pool_q8(const pkv_q8_pool* p, int32_t dtype) {
    return {p->k, p->v, p->k_scale, p->v_scale, p->num_blocks, p->block_size, p->num_kv_heads, p->head_dim, dtype};
}

}  // namespace

size_t pkv_chunk_workspace_bytes(const pkv_pool* pool, int32_t num_tokens, int32_t num_seqs,
                                 int32_t num_q_heads, int32_t max_context_len) {
    return pool ? chunk_workspace(chunk_pool(pool), num_tokens, num_seqs, num_q_heads, max_context_len) : 0;
}

pkv_status pkv_paged_attention_chunk(const pkv_pool* pool, const void* q, int32_t num_tokens,
                                     int32_t num_q_heads, const int32_t* query_start,
                                     int32_t num_seqs, const int32_t* block_tables,
                                     int32_t max_blocks_per_seq, const int32_t* context_lens,
                                     int32_t max_context_len, float scale, void* out,
                                     int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    const pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    return run_chunk(chunk_pool(pool), q, num_tokens, num_q_heads, query_start, num_seqs, block_tables,
                     max_blocks_per_seq, context_lens, max_context_len, scale, out, out_dtype, workspace,
                     workspace_bytes, stream);
}

namespace {

pkv_status check_q8(const pkv_q8_pool* pool, int32_t dtype) {
    if (!pool || !pool->k || !pool->v || !pool->k_scale || !pool->v_scale) return PKV_ERR_INVALID;
    if (!aligned16(pool->k) || !aligned16(pool->v) ||
        ((reinterpret_cast<uintptr_t>(pool->k_scale) | reinterpret_cast<uintptr_t>(pool->v_scale)) & 3u) != 0)
        return PKV_ERR_INVALID;
    if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->num_kv_heads <= 0 || pool->head_dim <= 0)
        return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID;
    if (dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
    if (pool->block_size != 16 && pool->block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (pool->head_dim != 64 && pool->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace

pkv_status pkv_qk_norm_rope_write_q8(const pkv_q8_pool* pool, int32_t dtype, const void* q,
                                     int64_t q_stride, const void* k, int64_t k_stride,
                                     const void* v, int64_t v_stride, int32_t num_tokens,
                                     int32_t num_q_heads, const void* q_weight,
                                     const void* k_weight, float eps, const float* cos_sin,
                                     int32_t max_position, int32_t rotary_dim, int32_t interleaved,
                                     const int32_t* positions, const int64_t* slot_mapping,
                                     void* q_out, void* stream) {
    pkv_status st = check_q8(pool, dtype);
    if (st != PKV_OK) return st;
    const int64_t pages = (int64_t)pool->num_blocks * pool->num_kv_heads;
    pkv::RopeParams p{};
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.num_kv_heads = pool->num_kv_heads;
    p.head_dim = pool->head_dim;
    st = rope_params(p, 2, pool->k, pool->v, pages * pool->block_size * pool->head_dim, q, q_stride, k, k_stride, v,
                     v_stride, num_tokens, num_q_heads, q_weight, k_weight, eps, cos_sin, max_position, rotary_dim,
                     interleaved, positions, slot_mapping, q_out);
    if (st != PKV_OK || num_tokens == 0) return st;
    const int64_t out_bytes = (int64_t)num_tokens * num_q_heads * pool->head_dim * 2;
    if (rows_overlap(pool->k_scale, pages * 4, pages * 4, 1, q_out, out_bytes) ||
        rows_overlap(pool->v_scale, pages * 4, pages * 4, 1, q_out, out_bytes))
        return PKV_ERR_INVALID;
    // what is written is written by many CTAs: no two of the four arrays share a byte
    const int64_t code_bytes = pages * pool->block_size * pool->head_dim;
    const void* const arrays[4] = {pool->k, pool->v, pool->k_scale, pool->v_scale};
    const int64_t bytes[4] = {code_bytes, code_bytes, pages * 4, pages * 4};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (rows_overlap(arrays[i], bytes[i], bytes[i], 1, arrays[j], bytes[j])) return PKV_ERR_INVALID;
    st = error_word(&p.err);
    if (st != PKV_OK) return st;
    return pkv::launch_q8_write(p, pool->k_scale, pool->v_scale, dtype, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

namespace {

struct Q8Layout {
    int32_t P, parts, column_tiles, clustered;
    size_t l_off, o_off, bytes;
};

// Maxima, sums and unscaled outputs of that many pieces' rows.
void q8_place(Q8Layout& w, size_t results, int32_t D) {
    w.l_off = (results * 4 + 15) & ~size_t(15);
    w.o_off = 2 * w.l_off;
    w.bytes = w.o_off + results * D * 4;
}

// How a decode call is cut.  A CTA has 8 columns (query, head) of a kv head, or 16: these share what is read and
// converted, but three fit an SM where four of the others do, and there are half as many.  16 are taken from
// about 2^20 tokens times tiles of 16 columns on (r below: that number over 2^20; 8 columns / 16, us):
//   32 heads of 128 on 8, 4 queries   16 requests of ~600 19.1 / 25.5 (r 0.2)    64 of ~600 43.3 / 41.2 (1.2)
//                                     64 of ~10,000 362 / 300 (20)
//   32 heads of 128 on 2              64 of ~600 17.9 / 25.7 (0.3)     64 of ~2500 33.7 / 32.3 (1.2)
//                                     256 of ~10,000 352 / 314 (20)
//   16 heads of 128 on 1              64 of ~10,000 50.5 / 55.3 (2.4)  256 of ~10,000 181 / 163 (10)
//   16 heads of 64 on 4, 4 queries    64 of ~600 18.6 / 19.4 (0.6)     64 of ~10,000 124 / 101 (10)
// Where SMs stay idle, a context is cut, so that there are four CTAs an SM: up to 4096 tokens into 8 pieces at
// most, which meet in a cluster, beyond into pieces of 128 to 1024 tokens.  No piece is shorter than 64 tokens
// (32 / 8 heads, 64 and 128: 1 request of 200 tokens 4.7 / 5.6 us, 8 of 80 5.3 / 4.9, others alike; 32 as 64).
// With pieces of up to 2048 instead of 1024 tokens 8 contexts of 60,000 take 161 and not 159 us, 2 of them 48 and
// not 52, and they end less together where lengths differ.
Q8Layout q8_layout(const pkv_q8_pool* pool, int32_t S, int32_t NQ, int32_t Hq, int32_t max_ctx, int32_t P) {
    const int64_t cols = (int64_t)NQ * (Hq / pool->num_kv_heads), rows = (int64_t)S * pool->num_kv_heads;
    Q8Layout w{};
    w.column_tiles = cols > 8 && rows * ((cols + 15) / 16) >= (1 << 20) / std::max(max_ctx, 1) ? 2 : 1;
    if (P > 0) {  // no more than the whole context
        const int64_t B = pool->block_size;
        w.P = (int32_t)std::min<int64_t>(P, (std::max<int64_t>(max_ctx, 1) + B - 1) / B * B);
    } else {
        const int64_t tile = 8 * w.column_tiles, ctas = std::max<int64_t>(1, rows * ((cols + tile - 1) / tile));
        const int64_t parts = std::max<int64_t>(1, 4 * (int64_t)sm_count() / ctas);
        int64_t x = std::max<int64_t>(64, ceil_div(max_ctx, parts));
        if (max_ctx <= 4096)
            x = std::max<int64_t>(x, ceil_div(max_ctx, pkv::Q8_CLUSTER));
        else
            x = std::min<int64_t>(std::max<int64_t>(x, 128), 1024);
        w.P = (int32_t)(ceil_div(x, pool->block_size) * pool->block_size);
    }
    w.parts = max_ctx > 0 ? ceil_div(max_ctx, w.P) : 1;
    w.clustered = w.parts > 1 && w.parts <= pkv::Q8_CLUSTER;
    if (w.parts <= 1 || w.clustered) return w;
    q8_place(w, (size_t)S * NQ * Hq * w.parts, pool->head_dim);
    return w;
}

// What a workspace has to hold for all calls up to this size whose pieces are chosen: contexts of more than
// 4096 tokens are cut into no more pieces than fill the SMs, 4 CTAs of at most 16 columns each (of which every
// one of their results is a row), or into pieces of 1024 tokens; and none is shorter than 128.
size_t q8_workspace(const pkv_q8_pool* pool, int32_t S, int32_t NQ, int32_t Hq, int32_t max_ctx) {
    if (max_ctx <= 4096) return 0;
    const size_t rows = (size_t)S * NQ * Hq;
    const int64_t cols = (int64_t)NQ * (Hq / pool->num_kv_heads);
    const size_t filling = (size_t)(4 * (int64_t)sm_count() * std::min<int64_t>(cols, 16));
    size_t results = std::min(rows * ceil_div(max_ctx, 128), filling);
    if (ceil_div(max_ctx, 1024) > pkv::Q8_CLUSTER) results = std::max(results, rows * ceil_div(max_ctx, 1024));
    Q8Layout w{};
    q8_place(w, results, pool->head_dim);
    return w.bytes;
}

}  // namespace

size_t pkv_decode_q8_workspace_bytes(const pkv_q8_pool* pool, int32_t num_seqs, int32_t num_queries,
                                     int32_t num_q_heads, int32_t max_context_len,
                                     int32_t partition_size) {
    if (!pool || pool->num_kv_heads <= 0 || pool->head_dim <= 0 || pool->block_size <= 0 || num_seqs < 0 ||
        num_queries <= 0 || num_q_heads <= 0 || max_context_len < 0 || partition_size < 0 ||
        num_q_heads % pool->num_kv_heads != 0)
        return 0;
    return partition_size > 0
               ? q8_layout(pool, num_seqs, num_queries, num_q_heads, max_context_len, partition_size).bytes
               : q8_workspace(pool, num_seqs, num_queries, num_q_heads, max_context_len);
}

pkv_status pkv_paged_attention_decode_q8(const pkv_q8_pool* pool, int32_t dtype, const void* q,
                                         int32_t num_queries, int32_t num_seqs,
                                         int32_t num_q_heads, const int32_t* block_tables,
                                         int32_t max_blocks_per_seq, const int32_t* context_lens,
                                         int32_t max_context_len, float scale, void* out,
                                         int32_t out_dtype, int32_t partition_size,
                                         void* workspace, size_t workspace_bytes, void* stream) {
    pkv_status st = check_q8(pool, dtype);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_queries <= 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
        num_q_heads % pool->num_kv_heads != 0 || !std::isfinite(scale) || partition_size < 0 ||
        partition_size % pool->block_size != 0)
        return PKV_ERR_INVALID;
    if (out_dtype != PKV_F32 && out_dtype != dtype) return PKV_ERR_UNSUPPORTED;
    const Q8Layout w = q8_layout(pool, num_seqs, num_queries, num_q_heads, max_context_len, partition_size);
    const int64_t cols = (int64_t)num_queries * (num_q_heads / pool->num_kv_heads);
    // (positions, with a piece added, are 32-bit numbers in the kernels)
    if (max_context_len > (1 << 30) || num_seqs > 65535 || w.parts > 65535 || cols > INT32_MAX - 8 ||
        pool->num_kv_heads * ((cols + 7) / 8) > INT32_MAX ||
        (int64_t)num_seqs * num_queries * num_q_heads > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !block_tables || !context_lens || !out || !aligned16(q) || !aligned16(out)) return PKV_ERR_INVALID;
    if (w.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < w.bytes)) return PKV_ERR_WORKSPACE;
    pkv::Q8DecodeParams p{};
    st = error_word(&p.err);
    if (st != PKV_OK) return st;
    p.k_pool = static_cast<const uint8_t*>(pool->k);
    p.v_pool = static_cast<const uint8_t*>(pool->v);
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.num_kv_heads = pool->num_kv_heads;
    p.q = q;
    p.num_seqs = num_seqs;
    p.num_queries = num_queries;
    p.num_q_heads = num_q_heads;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.partition_size = w.P;
    p.max_parts = w.parts;
    p.column_tiles = w.column_tiles;
    p.clustered = w.clustered;
    p.out = out;
    p.out_dtype = out_dtype;
    char* const ws = static_cast<char*>(workspace);
    p.part_m = reinterpret_cast<float*>(ws);
    p.part_l = reinterpret_cast<float*>(ws + w.l_off);
    p.part_o = reinterpret_cast<float*>(ws + w.o_off);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == PKV_F16 ? pkv::launch_q8_decode<__half>(p, pool->head_dim, s)
                                     : pkv::launch_q8_decode<__nv_bfloat16>(p, pool->head_dim, s);
    if (e == cudaSuccess && w.parts > 1 && !w.clustered) e = pkv::launch_q8_merge(p, pool->head_dim, s);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t pkv_chunk_q8_workspace_bytes(const pkv_q8_pool* pool, int32_t num_tokens, int32_t num_seqs,
                                    int32_t num_q_heads, int32_t max_context_len) {
    return pool ? chunk_workspace(chunk_pool_q8(pool, PKV_F16), num_tokens, num_seqs, num_q_heads, max_context_len) : 0;
}

pkv_status pkv_paged_attention_chunk_q8(const pkv_q8_pool* pool, int32_t dtype, const void* q,
                                        int32_t num_tokens, int32_t num_q_heads,
                                        const int32_t* query_start, int32_t num_seqs,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* context_lens, int32_t max_context_len,
                                        float scale, void* out, int32_t out_dtype, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    const pkv_status st = check_q8(pool, dtype);
    if (st != PKV_OK) return st;
    return run_chunk(chunk_pool_q8(pool, dtype), q, num_tokens, num_q_heads, query_start, num_seqs, block_tables,
                     max_blocks_per_seq, context_lens, max_context_len, scale, out, out_dtype, workspace,
                     workspace_bytes, stream);
}

pkv_status pkv_get_device_error(uint32_t* flags, void* stream) {
    if (!flags) return PKV_ERR_INVALID;
    unsigned int* err = nullptr;
    pkv_status st = error_word(&err);
    if (st != PKV_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int host = 0;
    if (cudaMemcpyAsync(&host, err, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemsetAsync(err, 0, sizeof(unsigned int), s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return PKV_ERR_CUDA;
    *flags = host;
    return host ? PKV_ERR_DEVICE : PKV_OK;
}

}  // extern "C"
