// Attention over a shared prefix, bf16: each request's own keys, the second launch of kda_prefix_attention.
//
// Bound by reading the own keys and values once.  Two ways to fill the GPU with that:
//   few requests   the work is cut along the keys as in the windowed attention's kernel for few rows: a cluster of
//                  up to 16 CTAs takes consecutive runs of 64-key tiles and joins them through distributed shared
//                  memory, in an order that the sizes alone decide
//   many           CTAs that stay take one (request, kv heads, rows) after the other, see below
// o (not divided), m and l of each row go to the workspace.
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
    int32_t G, kv_rows, page_shift;
    int32_t chunks;     // a cluster a chunk of rows (and further ones)
    int32_t heads;      // many requests: kv heads that a CTA takes at once
    float c;  // scale log2 e, > 0
};

struct Ring {
    uint64_t full[kStages], empty[kStages];
    int2 tile[kStages];       // first key; bit g: its keys 16 g .. have a page (and some row sees some)
    uint32_t abort;
    uint32_t busy;  // warps in own_rows, which may take longer than a wait does
};
struct Shared {
    Ring ring;
    float2 ml[kWarps][16];    // each warp's maximum reference and sum, by row
    uint32_t tainted;
};

__device__ __forceinline__ bool wait(Ring &ring, uint64_t *bar, uint32_t parity, const Params &p, uint32_t what) {
    return attn_wait_warp(bar, parity, &ring.abort, p.a, what, &ring.busy);
}

// The own keys of a chunk's rows: [from, last], tokens p0 .. last.
struct Own {
    int32_t from, p0, last;
    __device__ __forceinline__ bool visible(int32_t p, int32_t j) const { return j >= from && j <= p; }
    // Some row must not see some of the keys [j, j + n).
    __device__ __forceinline__ bool some_hidden(int32_t j, int32_t n) const { return j < from || j + (n - 1) > p0; }
};

// tma_load_box of what is read once: it is the first to leave L2, where the prefixes' tiles are read again and again.
__device__ __forceinline__ void load_once(uint32_t dst, const void *tmap, int y, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %2, %3, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(y), "r"(0), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// Fetches a tile, keys [j0, j0 + 64): whole pages (up to a tile), except that on an edge (j0 a multiple of 16, else
// of 64) only the groups of 16 keys come that some row sees.  n: tiles that went through the ring.
__device__ __forceinline__ bool produce(const Params &p, Ring &sh, unsigned char *sm, int32_t row, const Own &own, int32_t h,
                                        int32_t j0, bool edge, uint32_t &n) {
    const int lane = threadIdx.x & 31;
    const PrefixAttentionArgs &a = p.a;
    const int32_t page_shift = p.page_shift, s = n % kStages;
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    // lane b: box b of the tile
    const int32_t shift = edge ? 4 : min(page_shift, 6);
    const bool mine = lane << shift < kTile;
    const int32_t j = mine ? j0 + (lane << shift) : j0;
    int32_t id = -1;
    if (mine && (!edge || (j <= own.last && j + 15 >= own.from))) id = attn_page(a.cache, row, own.last, j >> page_shift);
    const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
    if (n >= kStages && !wait(sh, &sh.empty[s], (n / kStages - 1) & 1, p, 196)) return false;
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
        load_once(smem_u32(sm + s * kStageBytes + (lane << (shift + 9))), edge ? &p.tm_edge : &p.tm_kv, y, &sh.full[s], policy);
    }
    ++n;
    return true;
}
// Tiles [from, to) (numbers of 64-key tiles of the row).
__device__ __forceinline__ bool produce(const Params &p, Ring &sh, unsigned char *sm, int32_t row, const Own &own, int32_t h,
                                        int32_t from, int32_t to, uint32_t &n) {
    for (int32_t i = from; i < to; ++i)
        if (!produce(p, sh, sm, row, own, h, i * kTile, own.some_hidden(i * kTile, kTile), n)) return false;
    return true;
}
// Whichever warp gives up, the copies in flight (of tiles before n, from n0 on) land before the CTA leaves.
__device__ __forceinline__ void drain(Ring &sh, uint32_t n0, uint32_t n) {
    if ((threadIdx.x & 31) == 0)
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

// What a consumer warp holds of its 16 rows: this thread's are rows lane / 4 and lane / 4 + 8.
struct Rows {
    uint32_t q[8][4];
    float o[16][4], m[2], l[2];  // channels 8 t + 2 (lane % 4) + {0, 1} of either row
    int32_t pos[2];              // -1 sees nothing
    uint32_t bad;                // some value that not all rows of the item see is not finite
    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        bad = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
};

// q of rows row0 .. row0 + 15 (of num_rows) of a request and kv head.
__device__ __forceinline__ void load_q(const PrefixAttentionArgs &a, int32_t G, int32_t first, int32_t h, int32_t row0,
                                       int32_t num_rows, int32_t q0, Rows &w) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(a.q) + 2 * (lane & 3);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int32_t row = row0 + (lane >> 2) + 8 * u, token = row / G;
        const bool live = row < num_rows;
        w.pos[u] = live ? q0 + token : -1;
        const __nv_bfloat16 *src = base + ((int64_t)(first + (live ? token : 0)) * a.num_q_heads + h * G + (live ? row % G : 0)) * kD;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            w.q[s][u] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * s) : 0u;
            w.q[s][2 + u] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * s + 8) : 0u;
        }
    }
}

// A warp's share of the tile in stage s: all of it (kBlocks = kWarps; then steps that no row sees are passed over), or
// every key group of kWarps / kBlocks.
template <int kBlocks>
__device__ __forceinline__ void consume(const Params &p, const Ring &ring, unsigned char *sm, int32_t s, const Own &own, Rows &w) {
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr int kSteps = kTile / 16 * kBlocks / kWarps;  // steps of 16 keys of a warp
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / kBlocks;
    auto &q = w.q;
    auto &o = w.o;
    auto &m = w.m;
    auto &l = w.l;
    auto &pos = w.pos;
    const int2 info = ring.tile[s];
    const int32_t j0 = info.x;
    // some row must not see some key of the tile
    const bool masked = (info.y & 15) != 15 || own.some_hidden(j0, kTile);
    const uint32_t stage = smem_u32(sm + s * kStageBytes), shift = info.y >> 8, half_bytes = 128u << shift;
#pragma unroll (kBlocks == kWarps ? 1 : kSteps)
    for (int step = 0; step < kSteps; ++step) {
        const int key0 = 16 * (group * kSteps + step);  // of the tile
        if (kBlocks == kWarps && (j0 + key0 > own.last || j0 + key0 + 15 < own.from)) continue;
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
                    w.bad |= any_nonfinite(bm[t] & part[t & 1]);
                    bm[t] &= keep[t & 1];
                }
            }
            mma16816(o[2 * c], pr, bm[0], bm[1]);
            mma16816(o[2 * c + 1], pr, bm[2], bm[3]);
        }
    }
}

template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 2) prefix_own_kernel(const __grid_constant__ Params p) {
    constexpr int kRows = 16 * kBlocks;
    constexpr int kGroups = kWarps / kBlocks;         // key groups of a tile
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
            mbar_init(&sh.ring.full[i], 1);
            mbar_init(&sh.ring.empty[i], kWarps);
        }
        sh.ring.abort = sh.ring.busy = sh.tainted = 0;
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
            uint32_t n = n0;
            if (!attn_withhold(a)) produce(p, sh.ring, sm, req.row, own, h, from, to, n);
            drain(sh.ring, n0, n);
        } else {
            const int block = warp % kBlocks;
            Rows w;
            w.clear();
            load_q(a, G, req.first, h, row_base + 16 * block, num_rows, q0, w);
            uint32_t n = n0;
            for (int32_t i = from; i < to; ++i, ++n) {
                const int32_t s = n % kStages;
                if (!wait(sh.ring, &sh.ring.full[s], (n / kStages) & 1, p, 197)) break;
                consume<kBlocks>(p, sh.ring, sm, s, own, w);
                __syncwarp();
                if (lane == 0) arrive(&sh.ring.empty[s]);
            }
            if (w.bad) sh.tainted = 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                w.l[u] += __shfl_xor_sync(kAll, w.l[u], 1);
                w.l[u] += __shfl_xor_sync(kAll, w.l[u], 2);
                if ((lane & 3) == 0) sh.ml[warp][(lane >> 2) + 8 * u] = make_float2(w.m[u], w.l[u]);
            }
            // every consumer is past the ring's last tile: the partial outputs take its place
            asm volatile("bar.sync 1, 128;" ::: "memory");
            float *part = reinterpret_cast<float *>(sm) + warp * 16 * kPitch + (lane >> 2) * kPitch + 2 * (lane & 3);
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                *reinterpret_cast<float2 *>(part + 8 * t) = make_float2(w.o[t][0], w.o[t][1]);
                *reinterpret_cast<float2 *>(part + 8 * kPitch + 8 * t) = make_float2(w.o[t][2], w.o[t][3]);
            }
        }
        n0 += (uint32_t)(to - from);
        __syncwarp();
        cluster_sync();

        // Join: the rows go round the cluster's consumer warps, four channels a lane.
        bool failed = false, tainted = false;
        for (int32_t k = 0; k < splits; ++k) {
            failed |= remote_u32(remote(smem_u32(&sh.ring.abort), k)) != 0;
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
        // The partial outputs (plain stores) lie where the next rows' tiles go (TMA): the barrier orders the two only for those
        // who have said this.
        fence_proxy_async_smem();
        cluster_sync();  // the partials have been read: no CTA goes on to further rows, or leaves, before
        if (failed) break;
        if (threadIdx.x == 0) sh.tainted = 0;
        __syncthreads();
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) grid_wait();  // the launch ends after the one before it
}

// ---------------------------------------------------------------------------
// Many requests of a few rows a kv head each
// ---------------------------------------------------------------------------
// Here the CTAs (two an SM) stay and take work, kv heads of a request, as they get done, so that an item's beginning
// and end hide behind its neighbours' keys: a sixth warp takes the items, looks their requests up and brings q, and
// the fetching warp goes on to the next item's keys while the consumers end the last one's.  Which CTA computes an
// item makes no difference to it.  Own keys that fit in one tile
// go a warp a head (or row block), without a join.  256 requests of 1 to 2048 own keys (8 heads of 12 rows, 1.07 GB)
// take 182 us alone, 6.1 TB/s: HBM, and a tail of some 25 us while the last items end.  2,520 requests of 14 own keys
// in 4 heads: 69 us a call (a head at a time 123); there the time goes into items' beginnings and ends.
constexpr int kManyThreads = 32 * (kWarps + 2);
constexpr int kItems = 4;                      // in the queue
constexpr int kQPitch = 2 * kD + 16;           // bytes: the eight rows of a fragment in distinct banks
constexpr size_t kManyQ = kStages * kStageBytes, kManySwap = kManyQ + 16 * kQPitch;
constexpr size_t kManySmem = kManySwap + kWarps * 16 * 32 * sizeof(float) + 1024;

struct Item {
    int32_t first, base, rows;  // first token of the request; its rows base .. base + rows - 1 (0: no more items)
    int32_t table_row, q0;      // q0: index of the request's first token
    int32_t from, h;            // first own key, kv head
    // 0: the four warps share the keys of a block of 16 rows, or two and two those of two blocks.  Else all of the keys
    // are in one tile, from key() on, and a warp has a block of rows of one of the kv heads h .. h + heads - 1.
    int32_t heads;
    __device__ __forceinline__ Own own(int32_t G) const { return Own{from, q0 + base / G, q0 + (base + rows - 1) / G}; }
    __device__ __forceinline__ int32_t key() const { return from & ~15; }
};
struct ManyShared {
    Ring ring;
    uint64_t item_full[kItems], item_empty[kItems], q_full, q_empty;
    Item item[kItems];
    float2 ml[kWarps][16];
};

// Row r of an item, in kv head h, as a row of [T][Hq].
__device__ __forceinline__ int64_t place(const Params &p, const Item &it, int32_t h, int32_t r) {
    const int32_t row = it.base + r, token = row / p.G;
    return (int64_t)(it.first + token) * p.a.num_q_heads + h * p.G + (row - token * p.G);
}

// Rows r0, r0 + step .. below r1 of an item, in kv head h, by own_row (a row of 640,000 keys takes 0.6 s: the other warps'
// waits do not run out meanwhile).
__device__ __forceinline__ void own_rows(const Params &p, Ring &ring, const Item &it, int32_t h, const Own &own, int32_t r0, int32_t r1,
                                         int32_t step) {
    const int lane = threadIdx.x & 31;
    const PrefixSpace space = prefix_space(p.a);
    if (lane == 0) atomicAdd(&ring.busy, 1u);
    for (int32_t r = r0; r < r1; r += step) {
        float4 acc;
        const int64_t at = place(p, it, h, r);
        const float2 x = own_row(p, at, h, it.table_row, own, it.q0 + (it.base + r) / p.G, acc);
        store4(space.own_o + at * kD + 4 * lane, acc);
        if (lane == 0) space.own[at] = make_float4(x.x, x.y, it.from > 0, 0.f);
    }
    if (lane == 0) atomicSub(&ring.busy, 1u);
}

// Barrier 1 of the four consumer warps; whether any thread says x.
__device__ __forceinline__ bool consumers_or(bool x) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(any) : "r"((uint32_t)x) : "memory");
    return any != 0;
}

// The sixth warp.
template <int kRowBlocks, bool kShort>
__device__ void take_items(const Params &p, ManyShared &sh, unsigned char *sm, uint32_t *taken) {
    const int lane = threadIdx.x & 31;
    const PrefixAttentionArgs &a = p.a;
    // units: row blocks of heads of a request; those of the same heads run side by side and find the keys in L2
    const uint32_t parts = (uint32_t)(a.num_kv_heads / p.heads) * (uint32_t)p.chunks, units = (uint32_t)a.cache.batch * parts;
    uint32_t n = 0, with_q = 0;  // items published; those of one head
    const auto publish = [&](const Item &it) {
        const uint32_t s = n % kItems;
        if (n >= kItems && !wait(sh.ring, &sh.item_empty[s], (n / kItems - 1) & 1, p, 198)) return false;
        if (lane == 0) {
            sh.item[s] = it;
            arrive(&sh.item_full[s]);
        }
        __syncwarp();
        ++n;
        return true;
    };
    uint32_t ticket = 0;  // (lane 0's; on its way while the last one's items are published)
    if (lane == 0) ticket = atomicAdd(taken, 1u);
    while (true) {
        const uint32_t t = __shfl_sync(0xffffffffu, ticket, 0);
        if (t >= units) break;
        if (lane == 0) ticket = atomicAdd(taken, 1u);
        const uint32_t b = t / parts;
        const int32_t part = (int32_t)(t - b * parts), chunk = part % p.chunks, h0 = part / p.chunks * p.heads;
        const PrefixRequest req = prefix_request(a, p.cut, (int32_t)b);
        if (!req.ok && part == 0 && lane == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, b);
        const int32_t num_rows = req.n * p.G, step = 16 * kRowBlocks;
        for (int32_t base = step * chunk; base < num_rows; base += step * p.chunks) {
            Item it{req.first, base, min(step, num_rows - base), req.row, req.len - req.n, req.from, 0, 0};
            const int32_t blocks = (it.rows + 15) / 16;
            const bool short_keys = kShort && p.heads * blocks > 1 && it.own(p.G).last - it.key() < kTile;
            const int32_t each = short_keys ? kWarps / blocks : 1;  // heads of an item
            for (int32_t h = h0; h < h0 + p.heads; h += each) {
                it.h = h;
                it.heads = short_keys ? min(each, h0 + p.heads - h) : 0;
                if (!publish(it)) return;
                if (kRowBlocks > 1 || it.heads > 0) continue;
                uint4 x[8];  // rows lane / 16 + 2 i
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int32_t r = (lane >> 4) + 2 * i, token = (base + r) / p.G;
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < it.rows)
                        x[i] = *reinterpret_cast<const uint4 *>(
                            static_cast<const __nv_bfloat16 *>(a.q) +
                            ((int64_t)(req.first + token) * a.num_q_heads + h * p.G + base + r - token * p.G) * kD + 8 * (lane & 15));
                }
                if (with_q > 0 && !wait(sh.ring, &sh.q_empty, (with_q - 1) & 1, p, 199)) return;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(sm + kManyQ + ((lane >> 4) + 2 * i) * kQPitch + 16 * (lane & 15)) = x[i];
                __syncwarp();
                if (lane == 0) arrive(&sh.q_full);
                ++with_q;
            }
        }
    }
    publish(Item{});
}

// An item of two blocks of rows: consumer warps b and b + 2 share the keys of block b.  False: a wait gave up.
__device__ __forceinline__ bool two_blocks(const Params &p, ManyShared &sh, unsigned char *sm, const Item &it, uint32_t &tiles,
                                           Rows &w) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 1;
    const int32_t r0 = 16 * (warp & 1);
    const PrefixSpace space = prefix_space(p.a);
    const Own own = it.own(p.G);
    w.clear();
    load_q(p.a, p.G, it.first, it.h, it.base + r0, it.base + it.rows, it.q0, w);
    for (int32_t i = own.from / kTile; i <= own.last / kTile; ++i, ++tiles) {
        const int32_t st = tiles % kStages;
        if (!wait(sh.ring, &sh.ring.full[st], (tiles / kStages) & 1, p, 205)) break;
        consume<2>(p, sh.ring, sm, st, own, w);
        __syncwarp();
        if (lane == 0) arrive(&sh.ring.empty[st]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        w.l[u] += __shfl_xor_sync(0xffffffffu, w.l[u], 1);
        w.l[u] += __shfl_xor_sync(0xffffffffu, w.l[u], 2);
        if ((lane & 3) == 0) sh.ml[warp][(lane >> 2) + 8 * u] = make_float2(w.m[u], w.l[u]);
    }
    if (consumers_or(attn_given_up(&sh.ring.abort))) return false;
    if (consumers_or(w.bad != 0)) {
        own_rows(p, sh.ring, it, it.h, own, warp, it.rows, kWarps);
        return true;
    }
    float top[2], sum[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float2 x = sh.ml[warp & 1][(lane >> 2) + 8 * u], y = sh.ml[warp | 2][(lane >> 2) + 8 * u];
        top[u] = fmaxf(x.x, y.x);
        const auto weight = [&](float mx, float lx) {  // (a NaN sum stays one)
            return mx == -INFINITY ? (lx == 0.f ? 0.f : 1.f) : ex2_approx((mx - top[u]) * p.c);
        };
        sum[u] = fmaf(weight(y.x, y.y), y.y, weight(x.x, x.y) * x.y);
        const float mine = weight(w.m[u], w.l[u]);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            w.o[t][2 * u] *= mine;
            w.o[t][2 * u + 1] *= mine;
        }
    }
    // Each keeps half of the channels and gets the other's share of them, a quarter at a time.
    float4 *swap = reinterpret_cast<float4 *>(sm + kManySwap) + lane;  // [sender][4][lane]
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int a = 4 * turn + t, b = 8 + a;  // group 1's gift, group 0's
            swap[(warp * 4 + t) * 32] = group ? make_float4(w.o[a][0], w.o[a][1], w.o[a][2], w.o[a][3])
                                              : make_float4(w.o[b][0], w.o[b][1], w.o[b][2], w.o[b][3]);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float4 x = swap[((warp ^ 2) * 4 + t) * 32];
            const int a = 4 * turn + t, b = 8 + a;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w;
                if (group) w.o[b][e] += y;
                else w.o[a][e] += y;
            }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int32_t r = r0 + (lane >> 2) + 8 * u;
        if (r >= it.rows) continue;
        const int64_t at = place(p, it, it.h, r);
        float *o = space.own_o + at * kD + 64 * group + 2 * (lane & 3);
#pragma unroll
        for (int t = 0; t < 8; ++t)
            *reinterpret_cast<float2 *>(o + 8 * t) = group ? make_float2(w.o[8 + t][2 * u], w.o[8 + t][2 * u + 1])
                                                           : make_float2(w.o[t][2 * u], w.o[t][2 * u + 1]);
        if (group == 0 && (lane & 3) == 0) space.own[at] = make_float4(top[u], sum[u], it.from > 0, 0.f);
    }
    return true;
}

// An item of one block of rows: the four warps share its keys.  False: a wait gave up.
__device__ __forceinline__ bool one_block(const Params &p, ManyShared &sh, unsigned char *sm, const Item &it, uint32_t &tiles,
                                          Rows &w) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PrefixSpace space = prefix_space(p.a);
    {
        const uint32_t at = smem_u32(sm) + (uint32_t)kManyQ + (lane & 15) * kQPitch + 16 * (lane >> 4);
#pragma unroll
        for (int c = 0; c < 8; ++c) ldmatrix4(at + 32 * c, w.q[c]);
    }
    __syncwarp();
    if (lane == 0) arrive(&sh.q_empty);
    w.clear();
    const Own own = it.own(p.G);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int32_t r = (lane >> 2) + 8 * u;
        w.pos[u] = r < it.rows ? it.q0 + (it.base + r) / p.G : -1;
    }
    for (int32_t i = own.from / kTile; i <= own.last / kTile; ++i, ++tiles) {
        const int32_t st = tiles % kStages;
        if (!wait(sh.ring, &sh.ring.full[st], (tiles / kStages) & 1, p, 203)) break;
        consume<1>(p, sh.ring, sm, st, own, w);
        __syncwarp();
        if (lane == 0) arrive(&sh.ring.empty[st]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        w.l[u] += __shfl_xor_sync(kAll, w.l[u], 1);
        w.l[u] += __shfl_xor_sync(kAll, w.l[u], 2);
        if ((lane & 3) == 0) sh.ml[warp][(lane >> 2) + 8 * u] = make_float2(w.m[u], w.l[u]);
    }
    if (consumers_or(attn_given_up(&sh.ring.abort))) return false;  // (the rows have no result)
    if (consumers_or(w.bad != 0)) {
        own_rows(p, sh.ring, it, it.h, own, warp, it.rows, kWarps);
        return true;
    }
    // The warps' shares joined: warp w gets channels 32 w .. of every row from the other three, one after
    // the other through 8 KB, lane to lane.
    float top[2], sum[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float2 ml[kWarps];
        top[u] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            ml[k] = sh.ml[k][(lane >> 2) + 8 * u];
            top[u] = fmaxf(top[u], ml[k].x);
        }
        const auto weight = [&](float mx, float lx) {  // (a NaN sum stays one)
            return mx == -INFINITY ? (lx == 0.f ? 0.f : 1.f) : ex2_approx((mx - top[u]) * p.c);
        };
        sum[u] = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum[u] = fmaf(weight(ml[k].x, ml[k].y), ml[k].y, sum[u]);
        const float mine = weight(w.m[u], w.l[u]);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            w.o[t][2 * u] *= mine;
            w.o[t][2 * u + 1] *= mine;
        }
    }
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
        if (k == warp)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = make_float4(w.o[4 * k + t][0], w.o[4 * k + t][1], w.o[4 * k + t][2], w.o[4 * k + t][3]);
    float4 *swap = reinterpret_cast<float4 *>(sm + kManySwap) + lane;  // [receiver][4][lane]
#pragma unroll 1
    for (int turn = 1; turn < kWarps; ++turn) {
        const int to = (warp + turn) % kWarps;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            if (k == to)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    swap[(k * 4 + t) * 32] = make_float4(w.o[4 * k + t][0], w.o[4 * k + t][1], w.o[4 * k + t][2], w.o[4 * k + t][3]);
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float4 x = swap[(warp * 4 + t) * 32];
            acc[t] = make_float4(acc[t].x + x.x, acc[t].y + x.y, acc[t].z + x.z, acc[t].w + x.w);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int32_t r = (lane >> 2) + 8 * u;
        if (r >= it.rows) continue;
        const int64_t at = place(p, it, it.h, r);
        float *o = space.own_o + at * kD + 32 * warp + 2 * (lane & 3);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<float2 *>(o + 8 * t) = u ? make_float2(acc[t].z, acc[t].w) : make_float2(acc[t].x, acc[t].y);
        if (warp == 0 && (lane & 3) == 0) space.own[at] = make_float4(top[u], sum[u], it.from > 0, 0.f);
    }
    return true;
}

// Items of up to kRowBlocks blocks of rows; kShort: with items whose keys are all in one tile.  (Apart, since all of it
// together costs 16 x 4 beams 92 us instead of 80: instructions to fetch, and registers that spill.)
template <int kRowBlocks, bool kShort>
__global__ void __launch_bounds__(kManyThreads, 2) prefix_own_many_kernel(const __grid_constant__ Params p) {
    constexpr uint32_t kAll = 0xffffffffu;
    extern __shared__ unsigned char dyn[];
    __shared__ ManyShared sh;
    unsigned char *sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PrefixAttentionArgs &a = p.a;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.ring.full[i], 1);
            mbar_init(&sh.ring.empty[i], kWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kWarps + 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, kWarps);
        sh.ring.abort = sh.ring.busy = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join comes up when the last CTA has
    const PrefixSpace space = prefix_space(a);
    __syncthreads();

    if (warp == kWarps + 1) {
        take_items<kRowBlocks, kShort>(p, sh, sm, space.taken);
    } else if (warp == kWarps) {
        uint32_t tiles = 0;
        for (uint32_t n = 0; !attn_withhold(a); ++n) {
            const uint32_t s = n % kItems;
            if (!wait(sh.ring, &sh.item_full[s], (n / kItems) & 1, p, 200)) break;
            const Item it = sh.item[s];
            __syncwarp();
            if (lane == 0) arrive(&sh.item_empty[s]);
            if (it.rows == 0) break;
            const Own own = it.own(p.G);
            bool ok = true;
            if (it.heads == 0) ok = produce(p, sh.ring, sm, it.table_row, own, it.h, own.from / kTile, own.last / kTile + 1, tiles);
            for (int32_t i = 0; ok && i < it.heads; ++i)
                ok = produce(p, sh.ring, sm, it.table_row, own, it.h + i, it.key(), true, tiles);
            if (!ok) break;
        }
        drain(sh.ring, 0, tiles);
    } else {
        uint32_t tiles = 0, with_q = 0;
        Rows w;
        for (uint32_t n = 0;; ++n) {
            const uint32_t s = n % kItems;
            bool got = wait(sh.ring, &sh.item_full[s], (n / kItems) & 1, p, 201);
            const Item it = sh.item[s];
            __syncwarp();
            if (lane == 0) arrive(&sh.item_empty[s]);
            if (kShort && it.heads > 0) {
                // Everyone waits for every tile and frees it, so that none falls behind the ring.
                const Own own = it.own(p.G);
                const int32_t blocks = (it.rows + 15) / 16, head = warp / blocks, h = it.h + head;
                const int32_t r0 = 16 * (warp - head * blocks), r1 = min(r0 + 16, it.rows);
                const bool mine = got && head < it.heads;
                w.clear();
                if (mine) load_q(a, p.G, it.first, h, it.base + r0, it.base + it.rows, it.q0, w);
                for (int32_t i = 0; got && i < it.heads; ++i, ++tiles) {
                    const int32_t st = tiles % kStages;
                    if (!(got = wait(sh.ring, &sh.ring.full[st], (tiles / kStages) & 1, p, 204))) break;
                    if (mine && i == head) consume<kWarps>(p, sh.ring, sm, st, own, w);
                    __syncwarp();
                    if (lane == 0) arrive(&sh.ring.empty[st]);
                }
                if (consumers_or(!got)) break;
                if (!mine) continue;
                if (__any_sync(kAll, w.bad != 0)) {
                    own_rows(p, sh.ring, it, h, own, r0, r1, 1);
                    continue;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    w.l[u] += __shfl_xor_sync(kAll, w.l[u], 1);
                    w.l[u] += __shfl_xor_sync(kAll, w.l[u], 2);
                    const int32_t r = r0 + (lane >> 2) + 8 * u;
                    if (r >= r1) continue;
                    const int64_t at = place(p, it, h, r);
                    float *o = space.own_o + at * kD + 2 * (lane & 3);
#pragma unroll
                    for (int t = 0; t < 16; ++t) *reinterpret_cast<float2 *>(o + 8 * t) = make_float2(w.o[t][2 * u], w.o[t][2 * u + 1]);
                    if ((lane & 3) == 0) space.own[at] = make_float4(w.m[u], w.l[u], it.from > 0, 0.f);
                }
                continue;
            }
            if (kRowBlocks == 1 && got && it.rows > 0) got = wait(sh.ring, &sh.q_full, with_q++ & 1, p, 202);
            if (consumers_or(!got) || it.rows == 0) break;  // all four or none
            if constexpr (kRowBlocks == 2) {
                if (!two_blocks(p, sh, sm, it, tiles, w)) break;
            }
            if constexpr (kRowBlocks == 1) {
                if (!one_block(p, sh, sm, it, tiles, w)) break;
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) grid_wait();  // the launch ends after the one before it
}

template <int kBlocks>
cudaError_t launch(const Params &p, int splits, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)splits * p.a.cache.batch * p.chunks), (unsigned)p.a.num_kv_heads);
    return launch_clusters(prefix_own_kernel<kBlocks>, grid, splits, kThreads, kSmem, stream, p);
}

template <int kRowBlocks, bool kShort>
cudaError_t launch_many(const Params &p, unsigned ctas, cudaStream_t stream) {
    const cudaError_t e = allow_smem(prefix_own_many_kernel<kRowBlocks, kShort>, kManySmem);
    return e == cudaSuccess ? launch_serial(prefix_own_many_kernel<kRowBlocks, kShort>, dim3(ctas), kManyThreads, kManySmem, stream, p) : e;
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
    const int64_t average = (T + B - 1) / B * p.G;
    const int rows = most <= 16 || average <= 16 ? 16 : 32;
    const int64_t need = (most + rows - 1) / rows, share = (2 * average + rows - 1) / rows;
    p.chunks = (int32_t)(need < share ? need : share);
    // Split a request's keys over a cluster as far as the CTAs fit on half of the SMs (two an SM; the other half may
    // have prefixes for long, and a cluster only starts whole) and keep two tiles each, as far as the table's width can
    // tell (lengths are on the device: two requests of 16 own keys take 20.0 us in a table of 10 pages and 22.0 in one of
    // 512 or 16,384; 6 x 21 requests of 200 the same 2 us more).  Six prompts of one request: 30 us; 33 with clusters for all SMs; six prompts of 21 requests with
    // up to 2,100 own keys the other way round, 41.7 against 40.8.
    const int64_t tiles = ((int64_t)a.cache.table_width * a.cache.page_size + kTile - 1) / kTile;
    const int64_t ctas = B * a.num_kv_heads * p.chunks;
    int splits = 1;
    while (splits < kMaxSplits && ctas * splits <= device_sm_count() / 2 && tiles >= 4 * splits) splits *= 2;
    if (splits * B * p.chunks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    // From one item an SM on the CTAs stay.  2 prompts x 26 beams in 4 heads: 68 us, 72 with a CTA an item; with 126
    // long items (6 x 21 beams, one head) 52, and 41 in clusters.
    if (splits == 1 && ctas > device_sm_count() && ctas < 0x7fffffff) {
        const int64_t most_ctas = 2 * device_sm_count();
        // Heads one by one balance best (16 prompts x 4 beams: 80 us, 94 with short keys a warp a head); where each CTA
        // gets many, several at once (1,210 requests of 10 own keys, 8 heads: 78 us instead of 129, without prefixes).
        p.heads = 1;
        while (a.num_kv_heads % (2 * p.heads) == 0 && ctas >= 2 * p.heads * 4 * most_ctas) p.heads *= 2;
        const unsigned n = (unsigned)(ctas < most_ctas ? ctas : most_ctas);
        if (rows > 16) return launch_many<2, true>(p, n, stream);
        return p.heads > 1 ? launch_many<1, true>(p, n, stream) : launch_many<1, false>(p, n, stream);
    }
    return rows == 16 ? launch<1>(p, splits, stream) : launch<2>(p, splits, stream);
}

}  // namespace kda
