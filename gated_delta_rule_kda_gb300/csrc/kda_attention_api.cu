// C ABI of the paged-cache operators (norm + rotation + append, sliding-window attention, page
// management): argument validation on the host, then kernel launches.  Nothing here allocates.
#include <atomic>

#include "kda_common.cuh"

using namespace kda;

namespace {

#ifdef KDA_DEBUG
// Armed by kda_debug_inject_attention_timeout, consumed by the next kda_window_attention.
std::atomic<int> g_withhold_attention{0};
#endif

constexpr int64_t kInt32Max = 0x7fffffffLL;

bool aligned(const void *p, size_t align) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0;
}
bool aligned_or_null(const void *p, size_t align) { return p == nullptr || aligned(p, align); }
bool ok_dtype(kda_dtype d) { return d == KDA_BF16 || d == KDA_FP32; }
int64_t elem_bytes(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }
kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// The cache's sizes and pointers (the pool itself apart).
kda_status check_cache(const CacheArgs &c, int32_t num_kv_heads) {
    if (c.batch < 1 || c.num_pages < 1 || c.page_size < 1 || c.table_rows < 1 || c.table_width < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(c.page_table, 4) || !aligned(c.slot, 4) || !aligned(c.cu_tokens, 4) ||
        !aligned(c.kv_len, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
        return KDA_ERR_UNSUPPORTED;
    if ((int64_t)c.table_width * c.page_size > kInt32Max ||
        2 * (int64_t)c.num_pages * c.page_size > kInt32Max / num_kv_heads)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status norm_rope(NormRopeArgs &a, bool append, void *stream) {
    const int32_t T = a.cache.total_tokens;
    if (!ok_dtype(a.in_dtype) || !ok_dtype(a.out_dtype) || T < 0 || a.num_q_heads < 1 ||
        a.num_kv_heads < 1 || a.rotary_dim < 0 || a.rotary_dim > kD || (a.norm & ~1) ||
        (a.interleaved & ~1))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_or_null(a.q_weight, 16) || !aligned_or_null(a.k_weight, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    if (a.rotary_dim > 0 && (a.num_positions < 1 || !aligned(a.rope_table, 16)))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t vec = 16 / elem_bytes(a.in_dtype);
    const struct { const void *p; int64_t stride; int32_t heads; } in[3] = {
        {a.q, a.q_stride, a.num_q_heads}, {a.k, a.k_stride, a.num_kv_heads},
        {a.v, a.v_stride, a.num_kv_heads}};
    for (int i = 0; i < (append ? 3 : 2); ++i) {
        if (in[i].stride < (int64_t)in[i].heads * kD || in[i].stride % vec != 0)
            return KDA_ERR_INVALID_ARGUMENT;
        if (T > 0 && !aligned(in[i].p, 16)) return KDA_ERR_INVALID_ARGUMENT;
    }
    if (T > 0 && (!aligned(a.q_out, 16) || !(append || aligned(a.k_out, 16)) ||
                  (a.rotary_dim > 0 && !aligned(a.positions, 4))))
        return KDA_ERR_INVALID_ARGUMENT;
    if (append) {
        if (!aligned(a.kv_pool, 16)) return KDA_ERR_INVALID_ARGUMENT;
        const kda_status s = check_cache(a.cache, a.num_kv_heads);
        if (s != KDA_OK) return s;
    }
    if (a.rotary_dim % 16 != 0 ||
        (int64_t)T * ((int64_t)a.num_q_heads + 2 * (int64_t)a.num_kv_heads) > kInt32Max)
        return KDA_ERR_UNSUPPORTED;
    a.status = device_status();
    return from_cuda(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

bool ok_pool(int32_t num_layers, int32_t num_pages, int64_t page_bytes, const void *pool) {
    return num_layers >= 1 && num_pages >= 1 && page_bytes >= 16 && page_bytes % 16 == 0 &&
           aligned(pool, 16);
}

}  // namespace

extern "C" {

kda_status kda_qk_norm_rope(kda_dtype in_dtype, kda_dtype out_dtype, int32_t total_tokens,
                            int32_t num_q_heads, int32_t num_kv_heads, const void *q,
                            int64_t q_stride, const void *k, int64_t k_stride,
                            const float *q_weight, const float *k_weight, float eps, int32_t norm,
                            const float *rope_table, int32_t num_positions, int32_t rotary_dim,
                            int32_t interleaved, const int32_t *positions, void *q_out,
                            void *k_out, void *stream) {
    NormRopeArgs a{};
    a.in_dtype = in_dtype; a.out_dtype = out_dtype;
    a.num_q_heads = num_q_heads; a.num_kv_heads = num_kv_heads;
    a.q = q; a.q_stride = q_stride; a.k = k; a.k_stride = k_stride;
    a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps; a.norm = norm;
    a.rope_table = rope_table; a.num_positions = num_positions; a.rotary_dim = rotary_dim;
    a.interleaved = interleaved; a.positions = positions; a.q_out = q_out; a.k_out = k_out;
    a.cache.total_tokens = total_tokens;
    return norm_rope(a, false, stream);
}

kda_status kda_qk_norm_rope_append(kda_dtype in_dtype, kda_dtype out_dtype, int32_t batch,
                                   int32_t total_tokens, int32_t num_q_heads,
                                   int32_t num_kv_heads, const void *q, int64_t q_stride,
                                   const void *k, int64_t k_stride, const void *v,
                                   int64_t v_stride, const float *q_weight, const float *k_weight,
                                   float eps, int32_t norm, const float *rope_table,
                                   int32_t num_positions, int32_t rotary_dim, int32_t interleaved,
                                   const int32_t *positions, int32_t num_pages, int32_t page_size,
                                   int32_t table_rows, int32_t table_width,
                                   const int32_t *page_table, const int32_t *slot,
                                   const int32_t *cu_tokens, const int32_t *kv_len, void *kv_pool,
                                   void *q_out, void *stream) {
    NormRopeArgs a{};
    a.in_dtype = in_dtype; a.out_dtype = out_dtype;
    a.num_q_heads = num_q_heads; a.num_kv_heads = num_kv_heads;
    a.q = q; a.q_stride = q_stride; a.k = k; a.k_stride = k_stride; a.v = v; a.v_stride = v_stride;
    a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps; a.norm = norm;
    a.rope_table = rope_table; a.num_positions = num_positions; a.rotary_dim = rotary_dim;
    a.interleaved = interleaved; a.positions = positions; a.q_out = q_out; a.kv_pool = kv_pool;
    a.cache = CacheArgs{batch, total_tokens, num_pages, page_size, table_rows, table_width,
                        page_table, slot, cu_tokens, kv_len};
    return norm_rope(a, true, stream);
}

kda_status kda_window_attention(kda_dtype dtype, int32_t batch, int32_t total_tokens,
                                int32_t max_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t num_pages, int32_t page_size, int32_t table_rows,
                                int32_t table_width, int32_t window, int32_t sinks, const void *q,
                                const void *kv_pool, const int32_t *page_table,
                                const int32_t *slot, const int32_t *cu_tokens,
                                const int32_t *kv_len, float scale, void *o, void *stream) {
    if (!ok_dtype(dtype) || total_tokens < 0 || max_tokens < 1 || num_q_heads < 1 ||
        num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 || window < 1 || sinks < 0 ||
        !aligned(kv_pool, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    if (total_tokens > 0 && (!aligned(q, 16) || !aligned(o, 16))) return KDA_ERR_INVALID_ARGUMENT;
    const CacheArgs c{batch, total_tokens, num_pages, page_size, table_rows, table_width,
                      page_table, slot, cu_tokens, kv_len};
    const kda_status s = check_cache(c, num_kv_heads);
    if (s != KDA_OK) return s;
    if (num_q_heads / num_kv_heads > 128 || num_kv_heads > 65535 ||
        (int64_t)total_tokens * num_q_heads > kInt32Max)
        return KDA_ERR_UNSUPPORTED;
    WindowAttentionArgs a{dtype, max_tokens, num_q_heads, num_kv_heads, window, sinks, q, kv_pool,
                          scale, o, c, device_status()};
#ifdef KDA_DEBUG
    a.withhold = g_withhold_attention.exchange(0);
#endif
    return from_cuda(launch_window_attention(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_debug_inject_attention_timeout(void) {
#ifdef KDA_DEBUG
    g_withhold_attention.store(1);
    return KDA_OK;
#else
    return KDA_ERR_UNSUPPORTED;
#endif
}

kda_status kda_pages_copy(int32_t num_layers, int32_t num_pages, int64_t page_bytes, int32_t n,
                          const int32_t *src, const int32_t *dst, void *pool, void *stream) {
    if (!ok_pool(num_layers, num_pages, page_bytes, pool) || n < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (n > 0 && (!aligned(src, 4) || !aligned(dst, 4))) return KDA_ERR_INVALID_ARGUMENT;
    const PageMoves m{num_layers, num_pages, n, page_bytes, src, dst, nullptr, pool};
    return from_cuda(launch_pages_copy(m, static_cast<cudaStream_t>(stream)));
}

// 16 bytes for a count, then three int32 arrays of one entry per page or row.
size_t kda_pages_workspace_size(int32_t num_pages, int32_t table_rows) {
    if (num_pages < 1 || table_rows < 1) return 0;
    const size_t n = num_pages > table_rows ? num_pages : table_rows;
    return 16 + 3 * n * sizeof(int32_t);
}

kda_status kda_pages_fork(int32_t num_layers, int32_t num_pages, int64_t page_bytes,
                          int32_t page_size, int32_t table_rows, int32_t table_width,
                          int32_t num_forks, const int32_t *parent, const int32_t *child,
                          int32_t *page_table, int32_t *kv_len, void *pool, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (!ok_pool(num_layers, num_pages, page_bytes, pool) || page_size < 1 || table_rows < 1 ||
        table_width < 1 || num_forks < 0 || num_forks > table_rows || !aligned(page_table, 4) ||
        !aligned(kv_len, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (num_forks > 0 && (!aligned(parent, 4) || !aligned(child, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (num_pages > (1 << 20) || table_rows > (1 << 18) ||
        (int64_t)table_width * page_size > kInt32Max)
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16) || workspace_bytes < kda_pages_workspace_size(num_pages, table_rows))
        return KDA_ERR_WORKSPACE;
    int32_t *list = static_cast<int32_t *>(workspace) + 4;
    const size_t n = num_pages > table_rows ? num_pages : table_rows;
    PageForkArgs a{};
    a.free_list = list; a.src = list + n; a.dst = list + 2 * n;
    a.moves = PageMoves{num_layers, num_pages, num_forks, page_bytes, a.src, a.dst, nullptr, pool};
    a.page_size = page_size; a.table_rows = table_rows; a.table_width = table_width;
    a.parent = parent; a.child = child; a.page_table = page_table; a.kv_len = kv_len;
    a.status = device_status();
    return from_cuda(launch_pages_fork(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_pages_release(int32_t table_rows, int32_t table_width, int32_t page_size,
                             int32_t n, const int32_t *rows, int32_t window, int32_t sinks,
                             int32_t *page_table, int32_t *kv_len, void *stream) {
    if (table_rows < 1 || table_width < 1 || page_size < 1 || n < 0 || window < 0 || sinks < 0 ||
        !aligned(page_table, 4) || !aligned(kv_len, 4) || (n > 0 && !aligned(rows, 4)))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((int64_t)table_width * page_size > kInt32Max) return KDA_ERR_UNSUPPORTED;
    const PageReleaseArgs a{table_rows, table_width, page_size, n, window, sinks, rows, page_table,
                            kv_len, device_status()};
    return from_cuda(launch_pages_release(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_pages_compact(int32_t num_layers, int32_t num_pages, int64_t page_bytes,
                             int32_t table_rows, int32_t table_width, const int32_t *table_in,
                             int32_t *table_out, int32_t *num_live, void *pool, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (!ok_pool(num_layers, num_pages, page_bytes, pool) || table_rows < 1 || table_width < 1 ||
        !aligned(table_in, 4) || !aligned(table_out, 4) || !aligned(num_live, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t bytes = (size_t)table_rows * table_width * sizeof(int32_t);
    const uintptr_t x = reinterpret_cast<uintptr_t>(table_in), y = reinterpret_cast<uintptr_t>(table_out);
    if (x != y && x < y + bytes && y < x + bytes) return KDA_ERR_INVALID_ARGUMENT;
    if (num_pages > (1 << 20) || table_rows > (1 << 18)) return KDA_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16) || workspace_bytes < kda_pages_workspace_size(num_pages, table_rows))
        return KDA_ERR_WORKSPACE;
    int32_t *list = static_cast<int32_t *>(workspace) + 4;
    const size_t n = num_pages > table_rows ? num_pages : table_rows;
    PageCompactArgs a{};
    a.count = static_cast<int32_t *>(workspace);
    a.src = list; a.dst = list + n; a.remap = list + 2 * n;
    a.moves = PageMoves{num_layers, num_pages, 0, page_bytes, a.src, a.dst, a.count, pool};
    a.table_rows = table_rows; a.table_width = table_width;
    a.table_in = table_in; a.table_out = table_out; a.num_live = num_live;
    return from_cuda(launch_pages_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
