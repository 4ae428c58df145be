// Shared device helpers and launcher declarations of libkda (sm_103a).
#pragma once

#include <atomic>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

constexpr int kD = KDA_HEAD_DIM;  // d_k = d_v = 128

// Device status word: [0] = kda_status code, [1] = kernel-specific detail.
// The first writer wins (atomicCAS on [0]).
struct DeviceStatus {
    uint32_t *word;
};

__device__ __forceinline__ void record_status(DeviceStatus st, uint32_t code, uint32_t detail) {
    if (st.word == nullptr) return;
    if (atomicCAS(st.word, 0u, code) == 0u) atomicExch(st.word + 1, detail);
}

// Ask L2 to fetch [p, p + bytes) ahead of its use (bytes a multiple of 16; p must lie in an
// allocation the caller owns).  The one-CTA-per-unit decode kernels use it for the state of
// the unit one resident wave ahead, so that HBM keeps streaming while resident CTAs compute.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Streaming multiprocessors of the current device (cached per device; a racing first call
// stores the same value).
inline int device_sm_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
    int sms = cache[slot].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
            sms = 1;
        cache[slot].store(sms, std::memory_order_relaxed);
    }
    return sms;
}

// Launches that may come up while the kernel before them on the stream still drains (programmatic
// stream serialization): the kernel calls grid_wait() before it touches memory, which returns once
// everything before it is complete.  Takes one to two microseconds off a chain of short kernels.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A kernel whose dynamic shared memory may, with what it declares itself, pass the default 48 KB is given
// `most` (the largest size that any of its calls needs) once per call: the setting is the process's, so
// one that followed the call's own size could be lowered by another thread between setting and launch.
template <typename... Params>
cudaError_t allow_smem(void (*kernel)(Params...), size_t most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

template <typename... Params, typename... Args>
cudaError_t launch_serial(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                          const Args &...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float x) { *p = x; }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p) {
        return __bfloat162float(*p);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float x) {
        *p = __float2bfloat16_rn(x);
    }
};

// Load 4 consecutive elements (16-byte aligned for fp32, 8-byte for bf16).
__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    uint2 raw = *reinterpret_cast<const uint2 *>(p);
    __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162 *>(&raw.x);
    __nv_bfloat162 b = *reinterpret_cast<__nv_bfloat162 *>(&raw.y);
    float2 fa = __bfloat1622float2(a), fb = __bfloat1622float2(b);
    return make_float4(fa.x, fa.y, fb.x, fb.y);
}
__device__ __forceinline__ void store4(float *p, float4 x) {
    *reinterpret_cast<float4 *>(p) = x;
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y);
    __nv_bfloat162 b = __floats2bfloat162_rn(x.z, x.w);
    uint2 raw;
    raw.x = *reinterpret_cast<uint32_t *>(&a);
    raw.y = *reinterpret_cast<uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(p) = raw;
}

// ---------------------------------------------------------------------------
// Launcher argument blocks (host side).  Pointers are device pointers that the
// ABI layer has already validated.
// ---------------------------------------------------------------------------
struct DecodeArgs {
    kda_dtype in_dtype, out_dtype;
    int32_t batch, num_heads;
    const void *q, *k, *v;
    const float *log_alpha, *beta;
    int32_t head_decay;  // 1: log_alpha is [B][H], one decay per (request, head)
    int32_t prefetch_ahead;  // units between a CTA and the one whose state it prefetches (0: none)
    float *S;
    float scale;
    void *o;
    DeviceStatus status;
};

// The whole layer core for a few tokens per request from pooled recurrent and
// short-convolution states (speculative verify / replay at the layer level).
constexpr int kDecodeLayerMaxTokens = KDA_DECODE_LAYER_MAX_TOKENS;
struct DecodeLayerTokensArgs {
    int32_t batch, num_heads, pool_size, total_tokens;
    const __nv_bfloat16 *qp, *kp, *vp, *z, *beta_logit, *g;  // [T][H][128] ([T][H] for beta_logit)
    const float *conv_w, *A, *b;                            // [3][H*128][4], [H], [H][128] or null
    const int32_t *cu_tokens, *slot;                        // [B+1], [B]
    float *S_pool;                                          // [P][H][128][128]
    __nv_bfloat16 *conv_pool;                               // [P][3][3][H][128]
    int32_t write_back;
    float scale, l2_eps, rms_eps;
    kda_dtype out_dtype;
    void *o;                                                // [T][H][128]
    int32_t prefetch_ahead;  // units between a CTA and the one whose state it prefetches (0: none)
    DeviceStatus status;
};

// Several tokens per request from a pooled state: request b's tokens are rows
// [cu_tokens[b], cu_tokens[b+1]) of q, k, v, log_alpha, beta; its state is S_pool[slot[b]].
struct DecodeTokensArgs {
    kda_dtype in_dtype, out_dtype;
    int32_t batch, num_heads, pool_size, total_tokens;
    const void *q, *k, *v;                 // [T][H][128]
    const float *log_alpha, *beta;         // [T][H][128], [T][H]
    const int32_t *cu_tokens, *slot;       // [B+1], [B]
    float *S_pool;                         // [P][H][128][128]
    int32_t write_back;                    // 1: the final state goes back to the pool row
    float *S_final;                        // [B][H][128][128] or null
    float scale;
    void *o;                               // [T][H][128]
    int32_t prefetch_ahead;  // units between a CTA and the one whose state it prefetches (0: none)
    DeviceStatus status;
};

// State snapshots during a prefill: for sequence n, snapshot k (k = 0, 1, ...) is the state
// after its first (k + 1) * every tokens, written to states[(base[n] + k)][h][j][c] while
// k < base[n + 1] - base[n].  every == 0: none.
struct Checkpoints {
    int32_t every;
    const int32_t *base;
    float *states;
};

// One decode step of the whole layer core for a batch of requests whose recurrent state
// and short-convolution state live in pools indexed by slot.
struct DecodeLayerArgs {
    int32_t batch, num_heads, pool_size;
    const __nv_bfloat16 *qp, *kp, *vp, *z, *beta_logit, *g;  // [B][H][128] ([B][H] for beta_logit)
    const float *conv_w, *A, *b;                            // [3][H*128][4], [H], [H][128] or null
    const int32_t *slot;                                    // [B]
    float *S_pool;                                          // [P][H][128][128]
    __nv_bfloat16 *conv_pool;                               // [P][3][3][H][128]
    float scale, l2_eps, rms_eps;
    kda_dtype out_dtype;
    void *o;                                                // [B][H][128]
    int32_t prefetch_ahead;  // units between a CTA and the one whose state it prefetches (0: none)
    DeviceStatus status;
};

struct PrefillArgs {
    kda_dtype in_dtype, out_dtype;
    int32_t num_seqs, total_tokens, num_heads;
    const void *q, *k, *v;
    const float *log_alpha, *beta, *S0;
    const int32_t *cu_seqlens;
    float scale;
    void *o;
    float *S_final;
    void *workspace;
    size_t workspace_bytes;
    Checkpoints ckpt;
    int32_t head_decay;  // 1: log_alpha is [T][H], one decay per (token, head)
    int32_t unbounded;   // 1: any decay <= 0 (no -5 floor): chunks out of the tensor-core range
                         //    run token by token; fp32 inputs run the token-by-token kernel
    DeviceStatus status;
};

struct FrontendArgs {
    int32_t num_seqs, total_tokens, num_heads;
    const __nv_bfloat16 *qp, *kp, *vp, *z, *beta_logit;
    const float *conv_w, *A, *b;
    const int32_t *cu_seqlens;
    float l2_eps;
    kda_dtype out_dtype;
    void *q_hat, *k_hat, *v_out;
    float *log_alpha, *beta;
    int32_t unbounded_decay;  // 1: log_alpha = -e^A softplus(z + b) instead of -5 sigmoid(e^A (z + b))
};

struct GateArgs {
    int64_t num_rows;
    kda_dtype in_dtype, out_dtype;
    const void *o_tilde;
    const __nv_bfloat16 *g;
    float eps;
    void *out;
};

// One KDA layer core in a single tensor-core kernel (front end and gate fused).
struct LayerArgs {
    int32_t num_seqs, total_tokens, num_heads;
    const __nv_bfloat16 *qp, *kp, *vp, *z, *beta_logit, *g;
    const float *conv_w, *A, *b, *S0;
    const int32_t *cu_seqlens;
    float scale, l2_eps, rms_eps;
    kda_dtype out_dtype;
    void *o;
    float *S_final;
    Checkpoints ckpt;
    int32_t unbounded_decay;  // 1: log_alpha = -e^A softplus(z + b) (no floor), chunk fallback
    DeviceStatus status;
};

// Contents checks of prefill inputs (offsets monotonic, log alpha in [-5, 0]).
struct CheckArgs {
    int32_t num_seqs, total_tokens, num_heads, head_decay;
    const float *log_alpha;  // [T][H][128] ([T][H] with head_decay) or null
    const int32_t *cu_seqlens;
    DeviceStatus status;
};

// The paged key/value cache of the softmax-attention layers (kda.h): one layer's pool, the
// table of pages per row, and the requests of a step.
struct CacheArgs {
    int32_t batch, total_tokens, num_pages, page_size, table_rows, table_width;
    const int32_t *page_table, *slot, *cu_tokens, *kv_len;  // [R][M], [B], [B+1], [R]
};

// Queries and keys normed per head and rotated; k and v into the cache when kv_pool is set.
struct NormRopeArgs {
    kda_dtype in_dtype, out_dtype;
    int32_t num_q_heads, num_kv_heads;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from token to token
    const float *q_weight, *k_weight;      // [128] or null
    float eps;
    int32_t norm, interleaved, rotary_dim, num_positions;
    const float *rope_table;   // [num_positions][rotary_dim / 2][2]
    const int32_t *positions;  // [T]
    void *q_out, *k_out;       // [T][Hq][128], [T][Hkv][128] (without a cache)
    void *kv_pool;             // [P][2][Hkv][page_size][128] or null
    CacheArgs cache;           // total_tokens always; the rest with kv_pool
    DeviceStatus status;
};

struct WindowAttentionArgs {
    kda_dtype dtype;
    int32_t max_tokens, num_q_heads, num_kv_heads, window, sinks;
    const void *q, *kv_pool;  // [T][Hq][128], [P][2][Hkv][page_size][128]
    float scale;
    void *o;  // [T][Hq][128]
    CacheArgs cache;
    DeviceStatus status;
#ifdef KDA_DEBUG
    int32_t withhold;  // test-only: the load warps fetch nothing, and waits give up after 1 ms
#endif
};

// Moves of pages: pages dst[i] := pages src[i] of each layer, i < *count (or n when null).
struct PageMoves {
    int32_t num_layers, num_pages, n;
    int64_t page_bytes;
    const int32_t *src, *dst, *count;
    void *pool;
};
struct PageForkArgs {
    PageMoves moves;
    int32_t page_size, table_rows, table_width;
    const int32_t *parent, *child;
    int32_t *page_table, *kv_len;
    int32_t *free_list, *src, *dst;  // [F] each, in the workspace
    DeviceStatus status;
};
struct PageReleaseArgs {
    int32_t table_rows, table_width, page_size, n, window, sinks;
    const int32_t *rows;
    int32_t *page_table, *kv_len;
    DeviceStatus status;
};
struct PageCompactArgs {
    PageMoves moves;
    int32_t table_rows, table_width;
    const int32_t *table_in;
    int32_t *table_out, *num_live;
    int32_t *src, *dst, *remap, *count;  // [P] each and [1], in the workspace
};

// The current device's status word (null when it cannot be found).
DeviceStatus device_status();

cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, cudaStream_t stream);
cudaError_t launch_window_attention(const WindowAttentionArgs &a, cudaStream_t stream);
cudaError_t launch_pages_copy(const PageMoves &a, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageForkArgs &a, cudaStream_t stream);
cudaError_t launch_pages_release(const PageReleaseArgs &a, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageCompactArgs &a, cudaStream_t stream);
cudaError_t launch_check_prefill(const CheckArgs &a, cudaStream_t stream);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream);
cudaError_t launch_decode_layer(const DecodeLayerArgs &a, cudaStream_t stream);
cudaError_t launch_decode_tokens(const DecodeTokensArgs &a, cudaStream_t stream);
cudaError_t launch_decode_layer_tokens(const DecodeLayerTokensArgs &a, cudaStream_t stream);
cudaError_t launch_prefill_recurrent(const PrefillArgs &a, cudaStream_t stream);
cudaError_t launch_prefill_tc(const PrefillArgs &a, cudaStream_t stream);
cudaError_t launch_layer_tc(const LayerArgs &a, cudaStream_t stream);
cudaError_t launch_frontend(const FrontendArgs &a, cudaStream_t stream);
cudaError_t launch_output_gate(const GateArgs &a, cudaStream_t stream);

}  // namespace kda
