// Attention over a shared prefix, bf16: each request's own keys, the second launch of kda_prefix_attention.
//
// Bound by reading the own keys and values once, so the work is cut along the keys as in the windowed
// attention's kernel for few rows: a cluster of up to 16 CTAs takes consecutive runs of 64-key tiles and
// joins them through distributed shared memory, in an order that the sizes alone decide; o (not divided), m
// and l of each row go to the workspace.
//
// A row is a (token, query head of the group) pair; a CTA has up to 32 of them, in one or two blocks of 16,
// and goes on to further ones where a request has more.  A producer warp fetches k and v by TMA, page by
// page, into a ring of 32 KB stages; of the four others, warp w takes row block w % kBlocks and every key
// group w / kBlocks of a tile, in steps of 16 keys on the warp-wide tensor instruction (m16n8k16).  The
// running maximum moves lazily.  Scores, m, l and o are fp32; p is rounded to bf16 for its product (at most
// 2^-8 of each weight).
//
// It comes up as soon as the prefixes' launch has, on the SMs that that leaves free, and waits for it only to
// end after it.
#include "kda_attention_mma.cuh"
#include "kda_prefix_attention.cuh"

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
    PrefixAttentionArgs a;
    PrefixCut cut;
    int32_t G, kv_rows, page_shift, chunks;
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

// The own keys of a chunk's rows: [from, last], tokens p0 .. last.
struct Own {
    int32_t from, p0, last;
    __device__ __forceinline__ bool visible(int32_t p, int32_t j) const { return j >= from && j <= p; }
    // Some row must not see some of the keys [j, j + n).
    __device__ __forceinline__ bool some_hidden(int32_t j, int32_t n) const { return j < from || j + (n - 1) > p0; }
};

// Fetches tiles [from, to) (numbers of 64-key tiles of the row): whole pages (up to a tile), except that of a
// tile on an edge only the groups of 16 keys come that some row sees.  n0: tiles that went through the ring before.
__device__ void produce(const Params &p, Shared &sh, unsigned char *sm, int32_t row, const Own &own, int32_t h,
                        int32_t from, int32_t to, uint32_t n0) {
    const int lane = threadIdx.x & 31;
    const PrefixAttentionArgs &a = p.a;
    const int32_t page_shift = p.page_shift;
    uint32_t n = n0;
    for (int32_t i = from; i < to; ++i, ++n) {
        const int32_t s = n % kStages, j0 = i * kTile;
        const bool edge = own.some_hidden(j0, kTile);
        // lane b: box b of the tile
        const int32_t shift = edge ? 4 : min(page_shift, 6);
        const bool mine = lane << shift < kTile;
        const int32_t j = mine ? j0 + (lane << shift) : j0;
        int32_t id = -1;
        if (mine && (!edge || (j <= own.last && j + 15 >= own.from))) id = attn_page(a.cache, row, own.last, j >> page_shift);
        const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
        if (n >= kStages && !wait(sh, &sh.empty[s], (n / kStages - 1) & 1, p, 196)) break;
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
        for (uint32_t k = n > n0 + kStages ? n - kStages : n0; k < n; ++k)
            mbar_wait_bounded(&sh.full[k % kStages], (k / kStages) & 1, kAttnWaitNs);
}

// One row's own keys alone (query q_row of [T][Hq], index pos), fp32 throughout, a key at a time; a warp a row, four
// channels a lane.  Runs only where a value that some tokens of the step see and others do not is not finite.
__device__ __noinline__ float2 own_row(const Params &p, int64_t q_row, int32_t h, int32_t table_row, const Own &own,
                                       int32_t pos, float4 &o) {
    const PrefixAttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int32_t page = a.cache.page_size;
    const float4 q = load4(static_cast<const __nv_bfloat16 *>(a.q) + q_row * kD + 4 * lane);
    const int64_t kv_stride = (int64_t)a.num_kv_heads * page * kD;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int32_t j = own.from; j <= pos; ++j) {  // (pos < 2^31 - 1)
        const int32_t id = attn_page(a.cache, table_row, pos, j / page);
        if (id < 0) continue;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.kv_pool) + (int64_t)id * 2 * kv_stride +
                                   ((int64_t)h * page + j % page) * kD + 4 * lane;
        const float4 k = load4(src), v = load4(src + kv_stride);
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float top = fmaxf(m, s), keep = top == -INFINITY ? 1.f : ex2_approx((m - top) * p.c);
        const float e = s == -INFINITY ? 0.f : ex2_approx((s - top) * p.c);  // (a NaN score stays one)
        l = l * keep + e;
        o = make_float4(o.x * keep + e * v.x, o.y * keep + e * v.y, o.z * keep + e * v.z, o.w * keep + e * v.w);
        m = top;
    }
    return make_float2(m, l);
}

template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 2) prefix_own_kernel(const __grid_constant__ Params p) {
    constexpr int kRows = 16 * kBlocks;
    constexpr int kGroups = kWarps / kBlocks;         // key groups of a tile
    constexpr int kSteps = kTile / 16 / kGroups;      // steps of 16 keys of a warp in a tile
    constexpr uint32_t kAll = 0xffffffffu;
    extern __shared__ unsigned char dyn[];
    __shared__ Shared sh;
    unsigned char *sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PrefixAttentionArgs &a = p.a;
    const int32_t splits = (int32_t)cluster_size(), rank = (int32_t)cluster_rank(), h = blockIdx.y, G = p.G;
    const int32_t item = (int32_t)blockIdx.x / splits, b = item / p.chunks, chunk0 = item - b * p.chunks;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        sh.abort = sh.tainted = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join comes up when the last CTA has
    const PrefixRequest req = prefix_request(a, p.cut, b);
    if (!req.ok && rank == 0 && h == 0 && chunk0 == 0 && threadIdx.x == 0)
        record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)b);
    const PrefixSpace space = prefix_space(a);
    const int32_t num_rows = req.n * G, q0 = req.len - req.n;  // q0: index of the first token
    __syncthreads();

    uint32_t n0 = 0;  // tiles that went through the ring
    for (int32_t row_base = chunk0 * kRows; row_base < num_rows; row_base += p.chunks * kRows) {  // the same for the whole cluster
        const int32_t rows = min(kRows, num_rows - row_base);
        const Own own{req.from, q0 + row_base / G, q0 + (row_base + rows - 1) / G};
        const int32_t tile0 = own.from / kTile, tiles = own.last / kTile + 1 - tile0;
        const int32_t from = tile0 + (int32_t)((int64_t)tiles * rank / splits);
        const int32_t to = tile0 + (int32_t)((int64_t)tiles * (rank + 1) / splits);
        if (warp == kWarps) {
            if (!attn_withhold(a)) produce(p, sh, sm, req.row, own, h, from, to, n0);
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
                    const int32_t row = row_base + row0 + 8 * u, token = row / G;
                    const bool live = row < num_rows;
                    pos[u] = live ? q0 + token : -1;  // -1 sees nothing
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

            uint32_t n = n0;
            for (int32_t i = from; i < to; ++i, ++n) {
                const int32_t s = n % kStages;
                if (!wait(sh, &sh.full[s], (n / kStages) & 1, p, 197)) break;
                const int2 info = sh.tile[s];
                const int32_t j0 = info.x;
                // some row must not see some key of the tile
                const bool masked = (info.y & 15) != 15 || own.some_hidden(j0, kTile);
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
                            uint32_t bm[4];
                            ldmatrix4(k_addr + (c >> 2) * half_bytes + row * 128 + ((chunk ^ (row & 7)) << 4), bm);
                            mma16816(sc[0], q[c], bm[0], bm[1]);
                            mma16816(sc[1], q[c], bm[2], bm[3]);
                        }
                    }
                    uint32_t keep[2] = {kAll, kAll}, part[2] = {0u, 0u};
                    if (masked) {
                        const bool mapped = info.y >> (key0 / 16) & 1;
                        // this thread's keys: 8 t + 2 (lane % 4) + {0, 1}
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int32_t j = j0 + key0 + 8 * t + 2 * (lane & 3) + e;
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    if (!(mapped && own.visible(pos[u], j))) sc[t][2 * u + e] = -INFINITY;
                                // of the values: keys that no row of the chunk sees are cleared, those that some see
                                // are looked at
                                const bool some = j >= own.from && j <= own.last, all = some && j <= own.p0;
                                const uint32_t half = e ? 0xffff0000u : 0x0000ffffu;
                                if (!some) keep[t] &= ~half;
                                else if (!all) part[t] |= half;
                            }
                    }
                    float now[2], f[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        now[u] = fmaxf(fmaxf(sc[0][2 * u], sc[0][2 * u + 1]), fmaxf(sc[1][2 * u], sc[1][2 * u + 1]));
                        now[u] = fmaxf(now[u], __shfl_xor_sync(kAll, now[u], 1));
                        now[u] = fmaxf(now[u], __shfl_xor_sync(kAll, now[u], 2));
                    }
                    const bool move0 = (now[0] - m[0]) * p.c > 8.f, move1 = (now[1] - m[1]) * p.c > 8.f;
                    if (__any_sync(kAll, move0 || move1)) {
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
                        uint32_t bm[4];
                        ldmatrix4_trans(v_addr + (c >> 2) * half_bytes + row * 128 + ((chunk ^ (row & 7)) << 4), bm);
                        if (masked) {
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                bad_values |= any_nonfinite(bm[t] & part[t & 1]);
                                bm[t] &= keep[t & 1];
                            }
                        }
                        mma16816(o[2 * c], pr, bm[0], bm[1]);
                        mma16816(o[2 * c + 1], pr, bm[2], bm[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) arrive(&sh.empty[s]);
            }
            if (bad_values) sh.tainted = 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                l[u] += __shfl_xor_sync(kAll, l[u], 1);
                l[u] += __shfl_xor_sync(kAll, l[u], 2);
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
        n0 += (uint32_t)(to - from);
        __syncwarp();
        cluster_sync();

        // Join: the rows go round the cluster's consumer warps, four channels a lane.
        bool failed = false, tainted = false;
        for (int32_t k = 0; k < splits; ++k) {
            failed |= remote_u32(remote(smem_u32(&sh.abort), k)) != 0;
            tainted |= remote_u32(remote(smem_u32(&sh.tainted), k)) != 0;
        }
        if (warp < kWarps && !failed) {  // (else the rows have no result)
            for (int32_t row = rank * kWarps + warp; row < rows; row += splits * kWarps) {
                const int32_t block = row >> 4, rr = row & 15, token = (row_base + row) / G, head = (row_base + row) - token * G;
                const int64_t q_row = (int64_t)(req.first + token) * a.num_q_heads + h * G + head;
                const int32_t sources = splits * kGroups;  // at most 64: two a lane
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float top, sum;
                if (tainted) {
                    const float2 x = own_row(p, q_row, h, req.row, own, q0 + token, acc);
                    top = x.x;
                    sum = x.y;
                } else {
                    float2 ml[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int32_t i = lane + 32 * u;
                        ml[u] = make_float2(-INFINITY, 0.f);
                        if (i < sources) ml[u] = remote_float2(remote(smem_u32(&sh.ml[(i % kGroups) * kBlocks + block][rr]), i / kGroups));
                    }
                    top = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
                    float w[2];
                    sum = 0.f;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {  // (a NaN sum stays one)
                        w[u] = ml[u].x == -INFINITY ? (ml[u].y == 0.f ? 0.f : 1.f) : ex2_approx((ml[u].x - top) * p.c);
                        sum = fmaf(w[u], ml[u].y, sum);
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
                    const uint32_t mine = smem_u32(sm) + (block * 16 + rr) * kPitch * 4 + 16 * lane;
#pragma unroll 8
                    for (int32_t i = 0; i < sources; ++i) {
                        const float wi = __shfl_sync(kAll, i < 32 ? w[0] : w[1], i & 31);
                        const float4 x = remote_float4(remote(mine + (i % kGroups) * kBlocks * 16 * kPitch * 4, i / kGroups));
                        acc = make_float4(fmaf(wi, x.x, acc.x), fmaf(wi, x.y, acc.y), fmaf(wi, x.z, acc.z), fmaf(wi, x.w, acc.w));
                    }
                }
                store4(space.own_o + q_row * kD + 4 * lane, acc);
                if (lane == 0) space.own[q_row] = make_float4(top, sum, req.from > 0, 0.f);
            }
        }
        __syncwarp();
        cluster_sync();  // the partials have been read: no CTA goes on to further rows, or leaves, before
        if (failed) break;
        if (threadIdx.x == 0) sh.tainted = 0;
        __syncthreads();
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) grid_wait();  // the launch ends after the one before it
}

template <int kBlocks>
cudaError_t launch(const Params &p, int splits, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)splits * p.a.cache.batch * p.chunks), (unsigned)p.a.num_kv_heads);
    return launch_clusters(prefix_own_kernel<kBlocks>, grid, splits, kThreads, kSmem, stream, p);
}

}  // namespace

cudaError_t launch_prefix_own(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream) {
    Params p;
    p.a = a;
    p.cut = cut;
    p.G = a.num_q_heads / a.num_kv_heads;
    p.kv_rows = (int32_t)(2ll * a.cache.num_pages * a.num_kv_heads * a.cache.page_size);
    p.c = (float)((double)a.scale * 1.4426950408889634);
    p.page_shift = a.cache.page_size == 16 ? 4 : a.cache.page_size == 32 ? 5 : a.cache.page_size == 64 ? 6 : 7;
    if (!encode_kv_box_map(&p.tm_kv, a.kv_pool, a.cache, a.num_kv_heads, a.cache.page_size < kTile ? a.cache.page_size : kTile) ||
        !encode_kv_box_map(&p.tm_edge, a.kv_pool, a.cache, a.num_kv_heads, 16))
        return cudaErrorNotSupported;
    // Chunks of rows: as many as the longest request may need, though not many more than all of them have
    // (a request that brings most of the step's tokens takes several turns then).
    const int64_t T = a.cache.total_tokens, B = a.cache.batch;
    const int64_t most = (a.max_tokens < T ? a.max_tokens : T) * p.G;
    const int rows = most <= 16 ? 16 : 32;
    const int64_t need = (most + rows - 1) / rows, share = (2 * ((T + B - 1) / B) * p.G + rows - 1) / rows;
    p.chunks = (int32_t)(need < share ? need : share);
    // Split a request's keys over a cluster as far as the CTAs are all resident at once (two an SM) and keep two
    // tiles each, as far as the table's width can tell.
    const int64_t tiles = ((int64_t)a.cache.table_width * a.cache.page_size + kTile - 1) / kTile;
    const int64_t ctas = B * a.num_kv_heads * p.chunks;
    int splits = 1;
    while (splits < kMaxSplits && ctas * splits <= device_sm_count() && tiles >= 4 * splits) splits *= 2;
    if (splits * B * p.chunks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return rows == 16 ? launch<1>(p, splits, stream) : launch<2>(p, splits, stream);
}

}  // namespace kda
