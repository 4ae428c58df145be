// C ABI of the operators that decode the branches of a request (attention over a shared prefix, beam
// selection, beam reordering): argument validation on the host, then kernel launches.  Nothing here allocates.
#include <atomic>

#include "kda_common.cuh"

using namespace kda;

namespace {

#ifdef KDA_DEBUG
// Armed by kda_debug_inject_prefix_timeout, consumed by the next kda_prefix_attention.
std::atomic<int> g_withhold_prefix{0};
#endif

constexpr int64_t kInt32Max = 0x7fffffffLL;

bool aligned(const void *p, size_t align) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0;
}
kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
bool ok_dtype(kda_dtype d) { return d == KDA_BF16 || d == KDA_FP32; }

}  // namespace

extern "C" {

size_t kda_prefix_attention_workspace_size(kda_dtype dtype, int32_t batch, int32_t total_tokens,
                                           int32_t num_groups, int32_t num_q_heads,
                                           int32_t num_kv_heads) {
    if (!ok_dtype(dtype) || batch < 1 || total_tokens < 0 || num_groups < 1 || num_q_heads < 1 || num_kv_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > 128)
        return 0;
    return prefix_attention_workspace(dtype, batch, total_tokens, num_groups, num_q_heads, num_kv_heads);
}

kda_status kda_prefix_attention(kda_dtype dtype, int32_t batch, int32_t total_tokens,
                                int32_t max_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t num_pages, int32_t page_size, int32_t table_rows,
                                int32_t table_width, int32_t num_groups, const void *q,
                                const void *kv_pool, const int32_t *page_table,
                                const int32_t *slot, const int32_t *cu_tokens,
                                const int32_t *kv_len, const int32_t *cu_groups,
                                const int32_t *prefix_len, float scale, void *o, void *workspace,
                                size_t workspace_bytes, void *stream) {
    if (!ok_dtype(dtype) || batch < 1 || total_tokens < 0 || max_tokens < 1 || num_q_heads < 1 || num_kv_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || num_pages < 1 || page_size < 1 || table_rows < 1 || table_width < 1 ||
        num_groups < 1 || !aligned(kv_pool, 16) || !aligned(page_table, 4) || !aligned(slot, 4) ||
        !aligned(cu_tokens, 4) || !aligned(kv_len, 4) || !aligned(cu_groups, 4) || !aligned(prefix_len, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (total_tokens > 0 && (!aligned(q, 16) || !aligned(o, 16) || q == o)) return KDA_ERR_INVALID_ARGUMENT;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)table_width * page_size > kInt32Max - 127 ||
        2 * (int64_t)num_pages * page_size > kInt32Max / num_kv_heads || num_q_heads / num_kv_heads > 128 ||
        num_kv_heads > 65535 || (int64_t)total_tokens * num_q_heads > kInt32Max || batch > (1 << 20) ||
        num_groups > (1 << 20))
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16) ||
        workspace_bytes < prefix_attention_workspace(dtype, batch, total_tokens, num_groups, num_q_heads, num_kv_heads))
        return KDA_ERR_WORKSPACE;
    PrefixAttentionArgs a{};
    a.dtype = dtype;
    a.max_tokens = max_tokens; a.num_q_heads = num_q_heads; a.num_kv_heads = num_kv_heads; a.num_groups = num_groups;
    a.q = q; a.kv_pool = kv_pool; a.cu_groups = cu_groups; a.prefix_len = prefix_len;
    a.scale = scale; a.o = o;
    a.cache = CacheArgs{batch, total_tokens, num_pages, page_size, table_rows, table_width,
                        page_table, slot, cu_tokens, kv_len};
    a.workspace = workspace;
    a.status = device_status();
#ifdef KDA_DEBUG
    a.withhold = g_withhold_prefix.exchange(0);
#endif
    return from_cuda(launch_prefix_attention(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_debug_inject_prefix_timeout(void) {
#ifdef KDA_DEBUG
    g_withhold_prefix.store(1);
    return KDA_OK;
#else
    return KDA_ERR_UNSUPPORTED;
#endif
}

size_t kda_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    if (batch < 1 || beams < 1 || beams > KDA_MAX_BEAMS || vocab < 1 || choices < 1 || choices > KDA_MAX_BEAMS) return 0;
    return beam_select_workspace(batch, beams, vocab, choices);
}

kda_status kda_beam_select(kda_dtype dtype, int32_t batch, int32_t beams, int32_t vocab,
                           int32_t choices, const void *logits, int64_t row_stride,
                           const float *scores, const uint8_t *ended, int32_t end_token,
                           int32_t *parent, int32_t *token, float *score, uint8_t *ended_out,
                           void *workspace, size_t workspace_bytes, void *stream) {
    if (!ok_dtype(dtype) || batch < 1 || beams < 1 || vocab < 1 || choices < 1 || row_stride < vocab ||
        end_token < -1 || end_token >= vocab || (ended != nullptr && end_token < 0) ||
        !aligned(logits, dtype == KDA_BF16 ? 2 : 4) || !aligned(scores, 4) || !aligned(parent, 4) ||
        !aligned(token, 4) || !aligned(score, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (beams > KDA_MAX_BEAMS || choices > KDA_MAX_BEAMS || vocab > (1 << 21) || (int64_t)batch * beams > (1 << 20))
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16) || workspace_bytes < beam_select_workspace(batch, beams, vocab, choices))
        return KDA_ERR_WORKSPACE;
    const BeamSelectArgs a{dtype, batch, beams, vocab, choices, logits, row_stride, scores, ended,
                           end_token, parent, token, score, ended_out, workspace};
    return from_cuda(launch_beam_select(a, static_cast<cudaStream_t>(stream)));
}

size_t kda_beam_reorder_workspace_size(int32_t num_pages, int32_t num_rows) {
    return kda_pages_workspace_size(num_pages, num_rows);
}

kda_status kda_beam_reorder(int32_t batch, int32_t beams, int32_t num_rows, const int32_t *parent,
                            int32_t *slot, int32_t *src, int32_t *dst, int32_t num_layers,
                            int32_t num_pages, int64_t page_bytes, int32_t page_size,
                            int32_t table_width, int32_t *page_table, int32_t *kv_len, void *pool,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (batch < 1 || beams < 1 || num_rows < 1 || !aligned(parent, 4) || !aligned(slot, 4) || !aligned(src, 4) ||
        !aligned(dst, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const bool cache = page_table != nullptr;
    if (cache && (num_layers < 1 || num_pages < 1 || page_bytes < 16 || page_bytes % 16 != 0 || !aligned(pool, 16) ||
                  page_size < 1 || table_width < 1 || !aligned(page_table, 4) || !aligned(kv_len, 4)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (beams > KDA_MAX_BEAMS || num_rows > (1 << 18)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)batch * beams > num_rows) return KDA_ERR_INVALID_ARGUMENT;
    if (cache && (num_pages > (1 << 20) || (int64_t)table_width * page_size > kInt32Max)) return KDA_ERR_UNSUPPORTED;
    if (cache && (!aligned(workspace, 16) || workspace_bytes < kda_pages_workspace_size(num_pages, num_rows)))
        return KDA_ERR_WORKSPACE;
    const BeamPlanArgs plan{batch, beams, num_rows, parent, slot, src, dst, device_status()};
    if (!cache) return from_cuda(launch_beam_slots(plan, static_cast<cudaStream_t>(stream)));
    int32_t *list = static_cast<int32_t *>(workspace) + 4;
    const size_t n = num_pages > num_rows ? num_pages : num_rows;
    PageForkArgs a{};
    a.free_list = list; a.src = list + n; a.dst = list + 2 * n;
    a.moves = PageMoves{num_layers, num_pages, batch * beams, page_bytes, a.src, a.dst, nullptr, pool};
    a.page_size = page_size; a.table_rows = num_rows; a.table_width = table_width;
    a.parent = src; a.child = dst; a.page_table = page_table; a.kv_len = kv_len;
    a.status = plan.status;
    a.beams = plan;
    return from_cuda(launch_beam_reorder(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
