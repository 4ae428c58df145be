// What the kernels of kda_window_attention share: the requests of a step, and which keys the
// tokens of a work item can see.
#pragma once

#include <cuda.h>

#include "kda_common.cuh"
#include "tc_primitives.cuh"

namespace kda {

// One request of the step, checked: its tokens [first, first + n) of q and o, its row of the
// table, and the tokens in that row (n of them the step's own).
struct AttnRequest {
    int32_t b, first, n, row, len;
};

// Request b, with n = 0 when its slot, kv_len or token range is out of range (then *bad is set).
__device__ __forceinline__ AttnRequest attn_request(const WindowAttentionArgs &a, int32_t b, bool *bad) {
    const CacheArgs &c = a.cache;
    AttnRequest r{b, c.cu_tokens[b], 0, c.slot[b], 0};
    const int32_t end = c.cu_tokens[b + 1];
    bool ok = r.first >= 0 && end >= r.first && end <= c.total_tokens && end - r.first <= a.max_tokens &&
              (uint32_t)r.row < (uint32_t)c.table_rows;
    if (ok) {
        r.len = c.kv_len[r.row];
        ok = r.len >= 0 && r.len <= c.table_width * c.page_size;
    }
    if (ok) r.n = end - r.first;
    *bad = !ok;
    return r;
}

// Walks the work items of a step in order: request b has ceil(n_b per / tile) of them, where n_b
// tokens make n_b * per rows of `tile`.  A whole warp calls find() with non-decreasing items.
struct AttnWalk {
    int32_t base = 0;      // requests [base, base + 32) were looked at last
    int64_t before = 0;    // items of the requests before base

    // The request that holds `item` and the item's number in it; false past the last item.
    __device__ __forceinline__ bool find(const WindowAttentionArgs &a, int64_t item, int32_t per,
                                         int32_t tile, AttnRequest &req, int32_t &index) {
        const int lane = threadIdx.x & 31;
        for (; base < a.cache.batch; base += 32) {
            AttnRequest mine{0, 0, 0, 0, 0};
            if (base + lane < a.cache.batch) {
                bool bad;
                mine = attn_request(a, base + lane, &bad);
                if (bad) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)(base + lane));
            }
            const int64_t items = ((int64_t)mine.n * per + tile - 1) / tile;
            int64_t sum = items;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += y;
            }
            const uint32_t holds = __ballot_sync(0xffffffffu, item < before + sum);
            if (holds != 0) {
                const int src = __ffs(holds) - 1;
                req.b = __shfl_sync(0xffffffffu, mine.b, src);
                req.first = __shfl_sync(0xffffffffu, mine.first, src);
                req.n = __shfl_sync(0xffffffffu, mine.n, src);
                req.row = __shfl_sync(0xffffffffu, mine.row, src);
                req.len = __shfl_sync(0xffffffffu, mine.len, src);
                index = (int32_t)(item - before - __shfl_sync(0xffffffffu, sum - items, src));
                return true;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        return false;
    }
};

// Keys that the tokens p in [p_min, p_max] of a row of `len` tokens see: [0, sink_end) and
// [low, end), in tiles of `tile` keys: tiles [0, sink_tiles) and [low_tile, end_tile).  A row may be
// 2^31 - 1 tokens long, so ends are rounded up to tiles in unsigned numbers.
struct AttnKeys {
    int32_t sink_tiles, low_tile, end_tile;
    __device__ __forceinline__ AttnKeys(int32_t p_min, int32_t p_max, int32_t window, int32_t sinks,
                                        int32_t tile) {
        const int32_t end = max(p_max + 1, 0);
        const int32_t low = p_min < window ? 0 : p_min - window + 1;
        const auto tiles = [tile](int32_t n) { return (int32_t)(((uint32_t)n + tile - 1) / tile); };
        end_tile = tiles(end);
        sink_tiles = tiles(min(sinks, end));
        low_tile = min(max(low / tile, sink_tiles), max(end_tile, sink_tiles));
        end_tile = max(end_tile, low_tile);
    }
    __device__ __forceinline__ int32_t count() const { return sink_tiles + end_tile - low_tile; }
    __device__ __forceinline__ int32_t tile(int32_t i) const {
        return i < sink_tiles ? i : low_tile + i - sink_tiles;
    }
};

// Clusters and their distributed shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
// The address of this CTA's shared address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 remote_float2(uint32_t addr) {
    float2 x;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float4 remote_float4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}
__device__ __forceinline__ uint32_t remote_u32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}

constexpr uint64_t kAttnWaitNs = 2000000000ull;  // longest wait
__device__ __forceinline__ uint64_t attn_wait_ns(const WindowAttentionArgs &a) {
#ifdef KDA_DEBUG
    if (a.withhold) return 1000000ull;
#endif
    return kAttnWaitNs;
}
__device__ __forceinline__ bool attn_withhold(const WindowAttentionArgs &a) {
#ifdef KDA_DEBUG
    return a.withhold != 0;
#else
    return false;
#endif
}
// Waits that run out.  `abort` is the CTA's word: set by the first to give up, seen by the other waits.
__device__ __forceinline__ bool attn_given_up(const uint32_t *abort) {
    return *reinterpret_cast<const volatile uint32_t *>(abort) != 0;
}
__device__ __forceinline__ void attn_give_up(uint32_t *abort, const WindowAttentionArgs &a, uint32_t what) {
    atomicExch(abort, 1u);
    record_status(a.status, KDA_ERR_DEVICE_TIMEOUT, what);
}
// A whole warp waits for a phase, for attn_wait_ns() at most or until another has given up.  Every lane gets the
// same answer: what follows are full-mask exchanges and warp-wide instructions, which lanes that went
// different ways could never meet in again.
__device__ __forceinline__ bool attn_wait_warp(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                               const WindowAttentionArgs &a, uint32_t what) {
    constexpr uint32_t kAll = 0xffffffffu;
    bool done = tc::mbar_try_wait(bar, parity);
    if (__all_sync(kAll, done)) return true;
    const uint64_t t0 = tc::global_timer_ns();
    while (true) {
        for (int i = 0; i < 4; ++i) {
            done = done || tc::mbar_try_wait(bar, parity);
            if (__all_sync(kAll, done)) return true;
        }
        if (__any_sync(kAll, attn_given_up(abort))) return false;
        if (__any_sync(kAll, tc::global_timer_ns() - t0 > attn_wait_ns(a))) {
            if ((threadIdx.x & 31) == 0) attn_give_up(abort, a, what);
            return false;
        }
    }
}

// A launch of clusters of `size` CTAs along x (above 8: the non-portable size), which may come up early
// as launch_serial's do: the kernel calls grid_wait().
template <typename Kernel, typename... Args>
cudaError_t launch_clusters(Kernel kernel, dim3 grid, int size, int threads, size_t smem, cudaStream_t stream,
                            const Args &...args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && size > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Whether the token with index p sees key j (of a mapped page).
__device__ __forceinline__ bool attn_visible(int32_t p, int32_t j, int32_t window, int32_t sinks) {
    return j <= p && (p - j < window || j < sinks);
}

// Page i of a row of the table, or -1 where there is none or it starts past index `last`.
__device__ __forceinline__ int32_t attn_page(const CacheArgs &c, int32_t row, int32_t last, int32_t i) {
    if (i >= c.table_width || i * c.page_size > last) return -1;
    const int32_t id = c.page_table[(int64_t)row * c.table_width + i];
    return (uint32_t)id < (uint32_t)c.num_pages ? id : -1;
}

// Whether either of two packed bf16 values is an infinity or NaN.
__device__ __forceinline__ uint32_t any_nonfinite(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u) | ((x & 0x7f800000u) == 0x7f800000u);
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// One row (query q_row of [T][Hq], index pos) from its visible keys alone, fp32 throughout; a warp a
// row, four channels a lane.  Runs only where a masked tile held a non-finite value.  A key at a time, each
// waiting for the one before: 0.6 to 0.9 us a visible key (two tokens over 131,072 keys with a NaN in one kv
// head 114 ms, against 0.12 without), so it must stay as rare as that.
__device__ __noinline__ inline void attn_row(const WindowAttentionArgs &a, int64_t q_row, int32_t h,
                                             int32_t table_row, int32_t pos) {
    const int lane = threadIdx.x & 31;
    const int32_t page = a.cache.page_size;
    const int64_t row = q_row * kD + 4 * lane;
    const float4 q = load4(static_cast<const __nv_bfloat16 *>(a.q) + row);
    const int64_t kv_stride = (int64_t)a.num_kv_heads * page * kD;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int32_t j = 0; j <= pos; ++j) {
        if (!attn_visible(pos, j, a.window, a.sinks)) {
            j = max(j, pos - a.window);  // the gap between the sinks and the window
            continue;
        }
        const int32_t id = attn_page(a.cache, table_row, pos, j / page);
        if (id < 0) continue;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.kv_pool) + (int64_t)id * 2 * kv_stride +
                                   ((int64_t)h * page + j % page) * kD + 4 * lane;
        const float4 k = load4(src), v = load4(src + kv_stride);
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale;
        const float top = fmaxf(m, s), keep = top == -INFINITY ? 1.f : expf(m - top);
        const float e = s == -INFINITY ? 0.f : expf(s - top);  // (a NaN score stays one)
        l = l * keep + e;
        o = make_float4(o.x * keep + e * v.x, o.y * keep + e * v.y, o.z * keep + e * v.z, o.w * keep + e * v.w);
        m = top;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store4(static_cast<__nv_bfloat16 *>(a.o) + row, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

cudaError_t launch_window_attention_rows(const WindowAttentionArgs &a, cudaStream_t stream);
cudaError_t launch_window_attention_tc(const WindowAttentionArgs &a, cudaStream_t stream);
constexpr int kSplitRows = 32;  // most rows of a request and kv head that the split kernel takes
cudaError_t launch_window_attention_split(const WindowAttentionArgs &a, cudaStream_t stream);

// A tensor map over kv_pool as rows of 128 channels, 64 channels x box_rows a box, 128-byte swizzle.
bool encode_kv_map(CUtensorMap *m, const WindowAttentionArgs &a, int32_t box_rows);
// The same rows seen as [k, v][half][row][64 channels] from a key row on: a box is the two halves of
// box_rows keys, then those of their values.
bool encode_kv_box_map(CUtensorMap *m, const WindowAttentionArgs &a, int32_t box_rows);

}  // namespace kda
