// Sliding-window attention over the paged cache, in fp32 on the FMA units.
//
// A work item is 32 rows of one request and key/value head; a row is a (token, query head of the
// group) pair, so that the group's heads share each key and value; kda_attention_rows.cuh computes a
// tile of 64 keys.  At the end o / l   (l = 0: no key was visible, o = 0).
// Measured: 3 requests of 40 to 300 tokens, window 257 + 3, 6 and 2 heads: 28 us (64-row items 35, without
// clusters 38); 4 us of FMAs a key tile and CTA.
// With few items a cluster of CTAs shares each one's key tiles, and joins the partial results
// through distributed shared memory.
#include <cfloat>

#include "kda_attention_rows.cuh"
#include "kda_window_attention.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

using tc::smem_u32;

using rows::kPitch;
using rows::kRows;
using rows::kSmem;
using rows::kThreads;
using rows::kTile;
using rows::kWarps;
constexpr int kMaxSplits = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) attention_rows_kernel(const WindowAttentionArgs a, int32_t splits) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int32_t G = a.num_q_heads / a.num_kv_heads, h = blockIdx.y;
    const CacheArgs &cache = a.cache;

    grid_wait();
    AttnRequest req;
    int32_t index;
    AttnWalk walk;
    const int32_t rank = (int32_t)cluster_rank();  // a cluster is one item
    if (!walk.find(a, blockIdx.x / splits, G, kRows, req, index)) return;  // the same for the whole cluster
    const int32_t num_rows = req.n * G, r0 = index * kRows;
    const int32_t p0 = req.len - req.n;  // index of the request's first token
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);

    rows::load_q(tiles_of, [&](int r) -> const T * {
        const int32_t row = r0 + r;
        return row < num_rows ? q + ((int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G) * kD : nullptr;
    });

    int32_t p[4];  // indices of this thread's rows 4 ty + i (past the last row: -1 sees nothing)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t row = r0 + 4 * ty + i;
        p[i] = row < num_rows ? p0 + row / G : -1;
    }
    rows::State st;

    const AttnKeys keys(p0 + r0 / G, p0 + (min(r0 + kRows, num_rows) - 1) / G, a.window, a.sinks, kTile);
    const int32_t end = p0 + (min(r0 + kRows, num_rows) - 1) / G + 1;  // no row sees a key from here on
    const int32_t tiles = keys.count(), last = (int32_t)((int64_t)tiles * (rank + 1) / splits);
    for (int32_t it = (int32_t)((int64_t)tiles * rank / splits); it < last; ++it) {
        // end <= len <= table_width * page_size
        rows::tile(tiles_of, s_keys, st, pool, cache, a.num_kv_heads, h, req.row, keys.tile(it) * kTile, end, a.scale,
                   [&](int i, int32_t j) { return attn_visible(p[i], j, a.window, a.sinks); });
    }
    auto &o = st.o;
    auto &m = st.m;
    auto &l = st.l;
    float *sk = tiles_of.k;
    const int warp = tid >> 5;

    T *out = static_cast<T *>(a.o);
    if (splits == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t row = r0 + 4 * ty + i;
            if (row >= num_rows) continue;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            T *dst = out + ((int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G) * kD;
            store4(dst + 4 * tx, make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv));
            store4(dst + 64 + 4 * tx, make_float4(o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv));
        }
        return;
    }
    // The partial results take the place of k; the cluster's CTAs join kRows / splits rows each.
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float *dst = sk + (4 * ty + i) * kPitch;
        *reinterpret_cast<float4 *>(dst + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        *reinterpret_cast<float4 *>(dst + 64 + 4 * tx) = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
        if (tx == 0) *reinterpret_cast<float2 *>(dst + kD) = make_float2(m[i], l[i]);
    }
    cluster_sync();
    for (int32_t r = rank * (kRows / splits) + warp; r < (rank + 1) * (kRows / splits); r += kWarps) {
        const int32_t row = r0 + r, lane = tid & 31;
        if (row >= num_rows) break;
        const uint32_t mine = smem_u32(sk + r * kPitch);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < splits) ml = remote_float2(remote(mine + kD * 4, lane));
        float top = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : expf(ml.x - top);  // (a NaN sum stays one)
        float sum = w * ml.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t s = 0; s < splits; ++s) {
            const float ws = __shfl_sync(0xffffffffu, w, s);
            const float4 x = remote_float4(remote(mine + 16 * lane, s));
            acc = make_float4(fmaf(ws, x.x, acc.x), fmaf(ws, x.y, acc.y), fmaf(ws, x.z, acc.z), fmaf(ws, x.w, acc.w));
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4(out + ((int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G) * kD + 4 * lane,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
    cluster_sync();  // no CTA leaves while another reads its partials
}

template <typename T>
cudaError_t launch_rows(const WindowAttentionArgs &a, cudaStream_t stream) {
    // each request rounds up to whole items at most once
    const int64_t rows = (int64_t)a.cache.total_tokens * (a.num_q_heads / a.num_kv_heads);
    const int64_t items = (rows + kRows - 1) / kRows + a.cache.batch;
    // Split an item's keys over a cluster as far as the CTAs are all resident at once (two an SM) and
    // keep two tiles each.
    const int64_t reach = (int64_t)a.window + a.sinks + kRows, held = (int64_t)a.cache.table_width * a.cache.page_size;
    const int64_t tiles = ((reach < held ? reach : held) + kTile - 1) / kTile;
    int splits = 1;
    while (splits < kMaxSplits && items * a.num_kv_heads * splits <= device_sm_count() && tiles >= 4 * splits) splits *= 2;
    if (items * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_clusters(attention_rows_kernel<T>, dim3((unsigned)(items * splits), (unsigned)a.num_kv_heads), splits,
                           kThreads, kSmem, stream, a, (int32_t)splits);
}

}  // namespace

cudaError_t launch_window_attention_rows(const WindowAttentionArgs &a, cudaStream_t stream) {
    return a.dtype == KDA_BF16 ? launch_rows<__nv_bfloat16>(a, stream) : launch_rows<float>(a, stream);
}

cudaError_t launch_window_attention(const WindowAttentionArgs &a, cudaStream_t stream) {
    if (a.cache.total_tokens == 0) return cudaSuccess;
    // The tensor-core kernel keeps its running maximum on unscaled scores, in the order that a
    // positive scale leaves alone; any other scale (and fp32) runs on the FMA units.
    const bool tensor = a.dtype == KDA_BF16 && a.scale > 0.f && a.scale <= FLT_MAX;
    if (!tensor) return launch_window_attention_rows(a, stream);
    // Up to 32 rows a request and kv head go to the split kernel (which wants them in one grid of at
    // most 65535 requests); more make a 128-row tile worth its while.  Measured at 8 kv heads, 8 query
    // heads each, split / tensor-core kernel: 4 tokens (32 rows), 64 requests at window 1024: 72 / 87 us,
    // 4 requests over 60,000 keys: 160 / 343 us; 8 tokens (64 rows): 129 / 87 and 335 / 344 us.
    const int64_t rows = (int64_t)a.max_tokens * (a.num_q_heads / a.num_kv_heads);
    return rows <= kSplitRows && a.cache.batch <= 65535 ? launch_window_attention_split(a, stream)
                                                : launch_window_attention_tc(a, stream);
}

}  // namespace kda
