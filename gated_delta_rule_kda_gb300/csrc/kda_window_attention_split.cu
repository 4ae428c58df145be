// Sliding-window attention over the paged cache for steps of few rows (single tokens, the verify of a
// short draft), bf16: each request and key/value head is split over a cluster of CTAs.
//
// Bound by reading k and v once (at 12 query heads a kv head, 24 flops a byte), so the work is cut
// along the keys until the GPU is full: the CTAs of a cluster (up to 16) take consecutive runs of
// 64-key tiles, and join their partial results through distributed shared memory:
//   M = max m_i;  o = (sum_i 2^(c (m_i - M)) o_i) / (sum_i 2^(c (m_i - M)) l_i)
// in one launch, with no workspace, in an order that the sizes alone decide.
//
// A row is a (token, query head of the group) pair; max_tokens G <= 32 of them, in one or two blocks
// of 16.  A producer warp fetches k and v by TMA, page by page, into a ring of 32 KB stages; of the
// four others, warp w takes row block w % kBlocks and every key group w / kBlocks of a tile, in steps
// of 16 keys on the warp-wide tensor instruction (m16n8k16): with at most 32 rows the 128-row MMA would
// idle, and the fragments of the 16-row one stay in registers from scores to outputs.  The running
// maximum moves lazily, as in the prefill kernel.  Scores, m, l and o are fp32; p is rounded to bf16
// for its product (at most 2^-8 of each weight).
// Measured: one token for each of 256 requests (rows of 1 to 8192, window 1024 + 4, 96 and 8 heads) 178 us,
// 5.9 TB/s of seen keys and values (0.87 of the measured copy bandwidth); two tokens for each of 4 requests
// over 65,536 to 131,072 (64 and 8 heads) 237 us, 6.35 TB/s; one token of one request 9.5 us.  A copy for
// each half of a box's channels and for k and v apart: 196 and 294 us (the producer's loop sets the pace);
// whole pages on the edges: 184; L2 prefetches four tiles ahead: 224.
#include "kda_attention_mma.cuh"
#include "kda_window_attention.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kWarps = 4;                     // consumers; one more fetches
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kTile = 64;                     // keys of a tile
constexpr uint32_t kStageBytes = kTile * 512;  // boxes of rows, each [k, v][half][row][64 channels]
constexpr int kStages = 3;
constexpr int kMaxSplits = 16;
constexpr int kPitch = kD + 4;                // partial outputs: fragment stores hit distinct banks
constexpr size_t kSmem = kStages * kStageBytes + 1024;  // the start is rounded up to 1024 bytes

struct Params {
    // The pool as [k, v][half of the channels][row][64 channels], boxes of both halves of both:
    CUtensorMap tm_kv;    // of min(page_size, 64) rows
    CUtensorMap tm_edge;  // of 16 rows
    WindowAttentionArgs a;
    int32_t G, kv_rows, page_shift;
    float c;  // scale log2 e, > 0
};

struct Shared {
    uint64_t full[kStages], empty[kStages];
    int2 tile[kStages];       // first key; bit g: its keys 16 g .. have a page (and some row sees some)
    float2 ml[kWarps][16];    // each warp's maximum reference and sum, by row
    uint32_t abort, tainted;
};

__device__ __forceinline__ bool wait(Shared &sh, uint64_t *bar, uint32_t parity, const Params &p, uint32_t what) {
    return attn_wait_warp(bar, parity, &sh.abort, p.a, what);
}

// Whether some row of a request (tokens p0 .. last) must not see some of the keys [j, j + n).
__device__ __forceinline__ bool some_hidden(const WindowAttentionArgs &a, int32_t j, int32_t n, int32_t p0, int32_t last) {
    return j + (n - 1) > p0 || (last - j >= a.window && j + (n - 1) >= a.sinks);
}

// Fetches tiles [from, to) of the request's key tiles: whole pages (up to a tile), except that of a
// tile on an edge only the groups of 16 keys come that some row sees (a window of 1024 and 4 first
// tokens over pages of 64 would otherwise read 12 % more).
__device__ void produce(const Params &p, Shared &sh, unsigned char *sm, const AttnRequest &req, const AttnKeys &keys,
                        int32_t h, int32_t from, int32_t to) {
    const int lane = threadIdx.x & 31;
    const WindowAttentionArgs &a = p.a;
    const int32_t page_shift = p.page_shift, p0 = req.len - req.n, last = req.len - 1;
    int32_t i = from;
    for (; i < to; ++i) {
        const int32_t n = i - from, s = n % kStages, j0 = keys.tile(i) * kTile;
        const bool edge = some_hidden(a, j0, kTile, p0, last);
        // lane b: box b of the tile
        const int32_t shift = edge ? 4 : min(page_shift, 6);
        const bool mine = lane << shift < kTile;
        const int32_t j = mine ? j0 + (lane << shift) : j0;
        int32_t id = -1;
        if (mine && (!edge || (j <= last && (p0 - j - 16 < a.window - 1 || j < a.sinks))))
            id = attn_page(a.cache, req.row, last, j >> page_shift);
        const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
        if (n >= kStages && !wait(sh, &sh.empty[s], (n / kStages - 1) & 1, p, 96)) break;
        if (lane == 0) {
            // a bit for 16 keys
            const uint32_t bits = shift == 4   ? exist
                                  : shift == 5 ? (exist & 1) * 3 + (exist & 2) * 6
                                               : exist * 15;
            sh.tile[s] = make_int2(j0, (int)(bits | (uint32_t)shift << 8));
            mbar_arrive_expect_tx(&sh.full[s], kStageBytes);
        }
        __syncwarp();
        if (mine) {
            const int32_t y = id < 0 ? p.kv_rows  // out of range: zeros
                                     : ((id * 2 * a.num_kv_heads + h) << page_shift) + (j & ((1 << page_shift) - 1));
            tma_load_box(smem_u32(sm + s * kStageBytes + (lane << (shift + 9))), edge ? &p.tm_edge : &p.tm_kv, y, &sh.full[s]);
        }
    }
    // Whichever warp gives up, the copies in flight land before the CTA leaves.
    if (lane == 0)
        for (int32_t k = max(from, i - kStages); k < i; ++k)
            mbar_wait_bounded(&sh.full[(k - from) % kStages], ((k - from) / kStages) & 1, kAttnWaitNs);
}

template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 2) attention_split_kernel(const __grid_constant__ Params p) {
    constexpr int kGroups = kWarps / kBlocks;         // key groups of a tile
    constexpr int kSteps = kTile / 16 / kGroups;      // steps of 16 keys of a warp in a tile
    extern __shared__ unsigned char dyn[];
    __shared__ Shared sh;
    unsigned char *sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WindowAttentionArgs &a = p.a;
    const int32_t splits = gridDim.x, h = blockIdx.y, G = p.G;
    const int32_t rank = (int32_t)cluster_rank();  // = blockIdx.x: a cluster is one row of the grid

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        sh.abort = sh.tainted = 0;
        fence_mbar_init();
    }
    grid_wait();
    bool bad;
    const AttnRequest req = attn_request(a, (int32_t)blockIdx.z, &bad);
    if (bad && rank == 0 && h == 0 && threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, blockIdx.z);
    if (req.n == 0) return;  // the whole cluster
    __syncthreads();

    const int32_t p0 = req.len - req.n, rows = req.n * G;  // p0: index of the first token
    const AttnKeys keys(p0, req.len - 1, a.window, a.sinks, kTile);
    const int32_t tiles = keys.count();
    const int32_t from = (int32_t)((int64_t)tiles * rank / splits), to = (int32_t)((int64_t)tiles * (rank + 1) / splits);

    if (warp == kWarps) {
        if (!attn_withhold(a)) produce(p, sh, sm, req, keys, h, from, to);
    } else {
        const int block = warp % kBlocks, group = warp / kBlocks;
        // this thread's two rows: 16 block + lane / 4 (+ 8)
        const int32_t row0 = 16 * block + (lane >> 2);
        int32_t pos[2];
        uint32_t q[8][4];
        {
            const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(a.q) + 2 * (lane & 3);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int32_t row = row0 + 8 * u, token = row / G;
                const bool live = row < rows;
                pos[u] = live ? p0 + token : -1;  // -1 sees nothing
                const __nv_bfloat16 *src = base + ((int64_t)(req.first + (live ? token : 0)) * a.num_q_heads + h * G + (live ? row % G : 0)) * kD;
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    q[s][u] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * s) : 0u;
                    q[s][2 + u] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * s + 8) : 0u;
                }
            }
        }
        float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        uint32_t bad_values = 0;

        for (int32_t i = from; i < to; ++i) {
            const int32_t n = i - from, s = n % kStages;
            if (!wait(sh, &sh.full[s], (n / kStages) & 1, p, 97)) break;
            const int2 info = sh.tile[s];
            const int32_t j0 = info.x;
            // some row must not see some key of the tile
            const bool masked = (info.y & 15) != 15 || some_hidden(a, j0, kTile, p0, req.len - 1);
            const uint32_t stage = smem_u32(sm + s * kStageBytes), shift = info.y >> 8, half_bytes = 128u << shift;
#pragma unroll
            for (int step = 0; step < kSteps; ++step) {
                const int key0 = 16 * (group * kSteps + step);  // of the tile
                // its box, and its place in it
                const uint32_t k_addr = stage + ((key0 >> shift) << (shift + 9)) + ((key0 & ((1 << shift) - 1)) << 7);
                const uint32_t v_addr = k_addr + 2 * half_bytes;
                float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                {
                    // matrices: keys 0-7 / 8-15 x channels 0-7 / 8-15 of the step
                    const int row = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int chunk = 2 * (c & 3) + (lane >> 3 & 1);
                        uint32_t b[4];
                        ldmatrix4(k_addr + (c >> 2) * half_bytes + row * 128 + ((chunk ^ (row & 7)) << 4), b);
                        mma16816(sc[0], q[c], b[0], b[1]);
                        mma16816(sc[1], q[c], b[2], b[3]);
                    }
                }
                uint32_t keep[2] = {0xffffffffu, 0xffffffffu}, part[2] = {0u, 0u};
                if (masked) {
                    // this thread's keys: 8 t + 2 (lane % 4) + {0, 1}
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int kk = key0 + 8 * t + 2 * (lane & 3) + e;
                            const int32_t j = j0 + kk;
                            const bool mapped = info.y >> (key0 / 16) & 1;
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                if (!(mapped && attn_visible(pos[u], j, a.window, a.sinks))) sc[t][2 * u + e] = -INFINITY;
                            // of the values: keys that no row of the request sees are cleared, those
                            // that some see are looked at
                            const bool sink = j < a.sinks;
                            const bool some = j <= req.len - 1 && (sink || p0 - j < a.window);
                            const bool all = j <= p0 && (sink || req.len - 1 - j < a.window);
                            const uint32_t half = e ? 0xffff0000u : 0x0000ffffu;
                            if (!some) keep[t] &= ~half;
                            else if (!all) part[t] |= half;
                        }
                }
                float now[2], f[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    now[u] = fmaxf(fmaxf(sc[0][2 * u], sc[0][2 * u + 1]), fmaxf(sc[1][2 * u], sc[1][2 * u + 1]));
                    now[u] = fmaxf(now[u], __shfl_xor_sync(0xffffffffu, now[u], 1));
                    now[u] = fmaxf(now[u], __shfl_xor_sync(0xffffffffu, now[u], 2));
                }
                const bool move0 = (now[0] - m[0]) * p.c > 8.f, move1 = (now[1] - m[1]) * p.c > 8.f;
                if (__any_sync(0xffffffffu, move0 || move1)) {
                    f[0] = move0 ? ex2_approx((m[0] - now[0]) * p.c) : 1.f;
                    f[1] = move1 ? ex2_approx((m[1] - now[1]) * p.c) : 1.f;
                    if (move0) m[0] = now[0];
                    if (move1) m[1] = now[1];
                    l[0] *= f[0];
                    l[1] *= f[1];
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        o[t][0] *= f[0];
                        o[t][1] *= f[0];
                        o[t][2] *= f[1];
                        o[t][3] *= f[1];
                    }
                }
                uint32_t pr[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float base = m[u] == -INFINITY ? 0.f : -m[u] * p.c;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float x = ex2_approx(fmaf(sc[t][2 * u], p.c, base));
                        const float y = ex2_approx(fmaf(sc[t][2 * u + 1], p.c, base));
                        l[u] += x + y;
                        const __nv_bfloat162 hh = __floats2bfloat162_rn(x, y);
                        pr[2 * t + u] = *reinterpret_cast<const uint32_t *>(&hh);
                    }
                }
                // matrices: keys 0-7 / 8-15 x channels 0-7 / 8-15, transposed
                const int row = lane & 15;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int chunk = 2 * (c & 3) + (lane >> 4);
                    uint32_t b[4];
                    ldmatrix4_trans(v_addr + (c >> 2) * half_bytes + row * 128 + ((chunk ^ (row & 7)) << 4), b);
                    if (masked) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            bad_values |= any_nonfinite(b[t] & part[t & 1]);
                            b[t] &= keep[t & 1];
                        }
                    }
                    mma16816(o[2 * c], pr, b[0], b[1]);
                    mma16816(o[2 * c + 1], pr, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.empty[s]);
        }
        if (bad_values) sh.tainted = 1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
            if ((lane & 3) == 0) sh.ml[warp][(lane >> 2) + 8 * u] = make_float2(m[u], l[u]);
        }
        // every consumer is past the ring's last tile: the partial outputs take its place
        asm volatile("bar.sync 1, 128;" ::: "memory");
        float *part = reinterpret_cast<float *>(sm) + warp * 16 * kPitch + (lane >> 2) * kPitch + 2 * (lane & 3);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            *reinterpret_cast<float2 *>(part + 8 * t) = make_float2(o[t][0], o[t][1]);
            *reinterpret_cast<float2 *>(part + 8 * kPitch + 8 * t) = make_float2(o[t][2], o[t][3]);
        }
    }
    __syncwarp();
    cluster_sync();

    // Join: the rows go round the cluster's consumer warps, four channels a lane.
    bool failed = false;
    for (int32_t r = 0; r < splits; ++r) failed |= remote_u32(remote(smem_u32(&sh.abort), r)) != 0;
    if (warp < kWarps && !failed) {
        bool tainted = false;
        for (int32_t r = 0; r < splits; ++r) tainted |= remote_u32(remote(smem_u32(&sh.tainted), r)) != 0;
        for (int32_t row = rank * kWarps + warp; row < rows; row += splits * kWarps) {
            const int32_t block = row >> 4, rr = row & 15;
            const int64_t q_row = (int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G;
            if (tainted) {
                attn_row(a, q_row, h, req.row, p0 + row / G);
                continue;
            }
            const int32_t sources = splits * kGroups;  // at most 64: two a lane
            float2 ml[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int32_t i = lane + 32 * u;
                ml[u] = make_float2(-INFINITY, 0.f);
                if (i < sources) ml[u] = remote_float2(remote(smem_u32(&sh.ml[(i % kGroups) * kBlocks + block][rr]), i / kGroups));
            }
            float top = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            float w[2], sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                w[u] = ml[u].x == -INFINITY ? (ml[u].y == 0.f ? 0.f : 1.f) : ex2_approx((ml[u].x - top) * p.c);
                sum = fmaf(w[u], ml[u].y, sum);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t mine = smem_u32(sm) + (block * 16 + rr) * kPitch * 4 + 16 * lane;
#pragma unroll 8
            for (int32_t i = 0; i < sources; ++i) {
                const float wi = __shfl_sync(0xffffffffu, i < 32 ? w[0] : w[1], i & 31);
                const float4 x = remote_float4(remote(mine + (i % kGroups) * kBlocks * 16 * kPitch * 4, i / kGroups));
                acc = make_float4(fmaf(wi, x.x, acc.x), fmaf(wi, x.y, acc.y), fmaf(wi, x.z, acc.z), fmaf(wi, x.w, acc.w));
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store4(static_cast<__nv_bfloat16 *>(a.o) + q_row * kD + 4 * lane,
                   make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its partials
}

template <int kBlocks>
cudaError_t launch(const Params &p, int splits, cudaStream_t stream) {
    const dim3 grid((unsigned)splits, (unsigned)p.a.num_kv_heads, (unsigned)p.a.cache.batch);
    return launch_clusters(attention_split_kernel<kBlocks>, grid, splits, kThreads, kSmem, stream, p);
}

}  // namespace

cudaError_t launch_window_attention_split(const WindowAttentionArgs &a, cudaStream_t stream) {
    Params p;
    p.a = a;
    p.G = a.num_q_heads / a.num_kv_heads;
    p.kv_rows = (int32_t)(2ll * a.cache.num_pages * a.num_kv_heads * a.cache.page_size);
    p.c = (float)((double)a.scale * 1.4426950408889634);
    p.page_shift = a.cache.page_size == 16 ? 4 : a.cache.page_size == 32 ? 5 : a.cache.page_size == 64 ? 6 : 7;
    if (!encode_kv_box_map(&p.tm_kv, a.kv_pool, a.cache, a.num_kv_heads, a.cache.page_size < kTile ? a.cache.page_size : kTile) ||
        !encode_kv_box_map(&p.tm_edge, a.kv_pool, a.cache, a.num_kv_heads, 16))
        return cudaErrorNotSupported;
    // Split as far as the CTAs are all resident at once (two an SM) and keep two tiles each: a second,
    // part-filled wave costs more than the longer rows (four requests of up to 131072 keys, 8 kv
    // heads: 239 us with 256 CTAs, 270 with 512).
    const int64_t reach = (int64_t)a.window + a.max_tokens - 1 + a.sinks;  // keys of a request, at most
    const int64_t held = (int64_t)a.cache.table_width * a.cache.page_size;
    const int64_t tiles = ((reach < held ? reach : held) + kTile - 1) / kTile;
    const int64_t ctas = (int64_t)a.cache.batch * a.num_kv_heads;
    int splits = 1;
    while (splits < kMaxSplits && ctas * splits <= device_sm_count() && tiles >= 4 * splits) splits *= 2;
    const int64_t rows = (int64_t)a.max_tokens * p.G;
    return rows <= 16 ? launch<1>(p, splits, stream) : launch<kSplitRows / 16>(p, splits, stream);
}

}  // namespace kda
