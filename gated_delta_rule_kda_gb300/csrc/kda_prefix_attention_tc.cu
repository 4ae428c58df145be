// Attention over a shared prefix on the tensor cores (bf16): the prefixes' launch of kda_prefix_attention.
//
//   s = q k^T;  p = 2^(c s - c m), c = scale log2 e;  l += sum p;  o += p v
// for up to 2 x 128 rows of a group and kv head, (token, query head) pairs of all the group's requests, over a
// stretch of the prefix's tiles of 128 keys; o, m and l go to the workspace.  Every row sees every key of
// the prefix, so nothing is masked but keys behind its end in the last tile and pages that do not exist,
// alike for all rows; the values of those keys are cleared, since a product with p = 0 would still turn a
// NaN or infinity into NaN.  m follows the running maximum lazily (it moves only past 2^8 in p); p enters
// its product rounded to bf16, which costs at most 2^-8 of each weight; all else is fp32.
//
// One CTA an SM, each with a run of (item, key tile) units of equal length:
//   warp 8      TMA: q of the next item, then k, v tiles page by page into a ring of five 32 KB stages (groups
//               of 16 keys in a last tile; what lies behind the end is an out-of-range box, which reads as zeros)
//   warps 9, 10 issue the products of two engines (s and o of 128 rows each in TMEM).  With two row tiles an
//               engine takes one of them, and the two take turns: while one row tile's softmax runs, the tensor
//               core works on the other's.  With one row tile they take its key tiles alternately, each with
//               an o, m and l of its own, which are joined at the end: the chain from scores to outputs of one
//               tile is hidden by the other's
//   warps 0-7   softmax, a thread a row: warps 0-3 engine 0, warps 4-7 engine 1; the stores of o, m, l
//   warp 11     clears the values behind the prefix's end
// TMEM: s0, s1, o0, o1 of 128 columns each.  Bound: the tensor core where a group brings 256 rows or more to
// a kv head; HBM (each key read once a group) where it brings few.  A unit of 128 keys and 256 rows takes a CTA some
// 1.6 us, 10.5 TFLOP/s (82 % of the GEMM rate of its SM, 93 % of what that sustains); one of up to 128 rows 1.5 to 1.8 us,
// at 5.3 to 5.4 TB/s in all.  128 tokens behind 131,072 shared keys: 148 CTAs, 357 us for most and 378 for the last.
#include <cuda.h>

#include "kda_attention_tc.cuh"
#include "kda_prefix_attention.cuh"

namespace kda {
namespace {

using namespace tc;
using namespace attn_tc;

constexpr int kItems = 4;         // work items announced ahead
constexpr int kItemReaders = 11;  // warps that read them: softmax, MMA, clearing
constexpr int kTiles = 8;         // key tiles whose masks are kept

enum Bar {
    B_QFULL, B_QEMPTY, B_KVFULL, B_RAW = B_KVFULL + kStages, B_KVEMPTY = B_RAW + kStages,
    B_CLEAN = B_KVEMPTY + kStages,
    B_S = B_CLEAN + kStages, B_P = B_S + 2, B_O = B_P + 4, B_ITEM = B_O + 2, B_ITEMFREE = B_ITEM + kItems,
    B_DRAIN = B_ITEMFREE + kItems, B_TURN = B_DRAIN + 2, B_JOIN = B_TURN + 2, B_WEIGHTS, B_JOINED, B_COUNT
};

constexpr uint32_t SM_Q = 0, SM_KV = 2 * kTileBytes, SM_END = SM_KV + kStages * kTileBytes;
constexpr size_t SM_DYN = SM_END + 1024;  // the start is rounded up to 1024 bytes

struct Params {
    CUtensorMap tm_q;     // [T][Hq][128], boxes of tq tokens x G heads x 64 channels
    CUtensorMap tm_kv;    // [2 P Hkv page_size][128], boxes of a page x 64 channels
    CUtensorMap tm_edge;  // of 16 keys x 64 channels
    PrefixAttentionArgs a;
    PrefixCut cut;
    int32_t tq;          // tokens of a row tile
    uint32_t inv_g;      // ceil(2^16 / G): x / G = x inv_g >> 16 for x < 128
    int32_t kv_rows;     // 2 P Hkv page_size
    int32_t page_shift;  // log2 page_size
    float c;             // scale log2 e, > 0
};

// A stretch of an item, found by the TMA warp and left in shared memory for the others.
struct Item {
    int32_t goes_on, more;  // with an item that another CTA started; else: CTAs that go on with it
    int32_t first, tokens;  // its tokens: rows [first, first + tokens) of q
    int32_t h, row;         // kv head, row of the table
    int32_t len;            // of the prefix
    int32_t tile, n;        // key tiles [tile, tile + n); n < 0: no more items

    __device__ __forceinline__ int32_t key(int32_t i) const { return kTile * (tile + i); }
    __device__ __forceinline__ bool two(const Params &p) const { return tokens > p.tq; }  // a second row tile
    // Tile i ends behind the prefix.
    __device__ __forceinline__ bool tail(int32_t i) const { return len - key(i) < kTile; }
};

struct Shared {
    uint64_t bar[B_COUNT];
    Item items[kItems];
    uint4 mask[kTiles];       // by key tile % 8: a bit a key that is there
    uint32_t masked[kTiles];  // some key is not
    float2 ml[kTile];         // one row tile: engine 1's m, l; then the weights of both engines
    uint32_t tmem, abort;
    PrefixRun run;
    int64_t sums[2 * kThreads / 32];
};

// One thread waits for a phase, giving up after attn_wait_ns() or when another warp has given up.
__device__ __noinline__ bool wait_one_on(Shared &sh, int bar, uint32_t parity, const Params &p) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (mbar_try_wait(sh.bar + bar, parity)) return true;
        if (attn_given_up(&sh.abort)) return false;
        if (global_timer_ns() - t0 > attn_wait_ns(p.a)) {
            attn_give_up(&sh.abort, p.a, (uint32_t)(128 + bar));
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_one(Shared &sh, int bar, uint32_t parity, const Params &p) {
    return mbar_try_wait(sh.bar + bar, parity) || wait_one_on(sh, bar, parity, p);
}
// A warp does, all lanes to one verdict.
__device__ __noinline__ bool wait_on(Shared &sh, int bar, uint32_t parity, const Params &p) {
    return attn_wait_warp(sh.bar + bar, parity, &sh.abort, p.a, (uint32_t)(128 + bar));
}
__device__ __forceinline__ bool wait(Shared &sh, int bar, uint32_t parity, const Params &p) {
    return __all_sync(0xffffffffu, mbar_try_wait(sh.bar + bar, parity)) || wait_on(sh, bar, parity, p);
}
// (the softmax warps have no registers to spare for calls)
__device__ __forceinline__ bool wait_inline(Shared &sh, int bar, uint32_t parity, const Params &p) {
    return attn_wait_warp(sh.bar + bar, parity, &sh.abort, p.a, (uint32_t)(128 + bar));
}

// The items in turn, for the warps that read them.
struct Items {
    uint32_t k = 0;
    // The next item, in its place until done(); null after the last one or when a wait gave up.  A whole
    // warp calls it (kHow 2: a softmax warp), or (kHow 1) one thread for its warp.
    template <int kHow = 0>
    __device__ __forceinline__ const Item *next(Shared &sh, const Params &p) {
        const uint32_t slot = k % kItems, phase = k / kItems & 1;
        const bool there = kHow == 1   ? wait_one(sh, B_ITEM + slot, phase, p)
                           : kHow == 2 ? wait_inline(sh, B_ITEM + slot, phase, p)
                                       : wait(sh, B_ITEM + slot, phase, p);
        if (!there) return nullptr;
        ++k;
        return sh.items[slot].n >= 0 ? &sh.items[slot] : nullptr;
    }
    __device__ __forceinline__ uint32_t slot() const { return (k - 1) % kItems; }
    // By one thread of the warp, which has read all it wants.
    __device__ __forceinline__ void done(Shared &sh) { mbar_arrive(sh.bar + B_ITEMFREE + slot()); }
};

// ---------------------------------------------------------------------------
// TMA
// ---------------------------------------------------------------------------
__device__ void tma_warp(const Params &p, Shared &sh, unsigned char *sm) {
    const int lane = threadIdx.x & 31;
    Ring ring;
    uint32_t loads = 0, items = 0, tiles = 0, uses[2] = {0, 0};  // bit s: parity of the uses of KVFULL, RAW + s
    bool ok = true;
    const auto load_item = [&](const Item &it) {
        const bool two = it.two(p);
        const auto load_q = [&] {  // when the last item's scores are done
            if (items > 0 && !wait(sh, B_QEMPTY, (items - 1) & 1, p)) return false;
            ++items;
            if (lane != 0) return true;
            const uint32_t bytes = (uint32_t)(p.tq * p.cut.G * 64 * 2);
            mbar_arrive_expect_tx(sh.bar + B_QFULL, bytes * (two ? 4u : 2u));
            for (int r = 0; r < (two ? 2 : 1); ++r)
                for (int half = 0; half < 2; ++half)
                    tma_load_3d(smem_u32(sm + SM_Q + r * kTileBytes + half * (kTileBytes / 2)), &p.tm_q,
                                64 * half, it.h * p.cut.G, it.first + r * p.tq, sh.bar + B_QFULL);
            return true;
        };
        // lane = 2 box + half: 64 channels of a page, or of 16 keys in a last tile.  The page of a tile's box is looked
        // up while the tile before is under way.
        const auto page_of = [&](int32_t i) {
            if (i >= it.n) return -1;
            const int32_t shift = it.tail(i) ? 4 : p.page_shift, j = it.key(i) + (lane >> 1 << shift);
            const bool mine = lane < 2 * kTile >> shift && j < it.len;
            return mine ? attn_page(p.a.cache, it.row, it.len - 1, j >> p.page_shift) : -1;
        };
        int32_t next = page_of(0);
        for (int32_t i = 0; ok && i < it.n; ++i) {
            const int32_t j0 = it.key(i);
            const bool tail = it.tail(i);
            const int32_t shift = tail ? 4 : p.page_shift, j = j0 + (lane >> 1 << shift);
            const bool mine = lane < 2 * kTile >> shift;
            const int32_t id = next;
            next = page_of(i + 1);
            const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
            for (int kv = 0; kv < 2; ++kv) {
                if (loads >= kStages && !(ok = wait(sh, B_KVEMPTY + ring.stage, ring.phase ^ 1, p))) break;
                const int raw = kv == 1 && tail ? 1 : 0;
                uint64_t *full = sh.bar + (raw ? B_RAW : B_KVFULL) + ring.stage;
                uses[raw] ^= 1u << ring.stage;
                if (lane == 0) {
                    if (kv == 0) {  // at most three tiles are ahead of a softmax: eight places do
                        uint32_t bits[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            bits[c] = low_bits(it.len - j0 - 32 * c);
                            if (shift == 4)
                                bits[c] &= (exist >> (4 * c) & 1 ? 0xffffu : 0u) | (exist >> (4 * c + 2) & 1 ? 0xffff0000u : 0u);
                            else if (!(exist >> (2 * (32 * c >> shift)) & 1)) bits[c] = 0;
                        }
                        sh.mask[tiles % kTiles] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
                        sh.masked[tiles % kTiles] = (bits[0] & bits[1] & bits[2] & bits[3]) != 0xffffffffu;
                    }
                    mbar_arrive_expect_tx(full, kTileBytes);
                }
                __syncwarp();
                if (mine) {
                    const int32_t y = id < 0 ? p.kv_rows  // out of range: zeros
                                             : (((id * 2 + kv) * p.a.num_kv_heads + it.h) << p.page_shift) +
                                                   (j & ((1 << p.page_shift) - 1));
                    tma_load_2d(smem_u32(sm + SM_KV + ring.stage * kTileBytes + (lane & 1) * (kTileBytes / 2) +
                                         ((lane >> 1) << (shift + 7))),
                                tail ? &p.tm_edge : &p.tm_kv, 64 * (lane & 1), y, full);
                }
                ring.next();
                ++loads;
                if (i == 0 && kv == 0 && !(ok = load_q())) break;  // q behind the first keys
            }
            ++tiles;
        }
        return ok;
    };
    PrefixWalk walk(sh.run);
    PrefixStretch s;
    bool more = true;
    for (uint32_t k = 0; ok && more; ++k) {
        more = walk.next(p.a, p.cut, sh.run, s);
        Item it;
        it.n = -1;
        if (more) {
            const int32_t t0 = s.index * p.cut.tile;
            it.goes_on = s.goes_on;
            it.more = s.more;
            it.first = s.first + t0;
            it.tokens = min(p.cut.tile, s.tokens - t0);
            it.h = s.h;
            it.row = s.row;
            it.len = s.len;
            it.tile = s.tile;
            it.n = s.count;
        }
        if (k >= kItems && !(ok = wait(sh, B_ITEMFREE + k % kItems, (k / kItems - 1) & 1, p))) break;
        if (lane == 0) {
            sh.items[k % kItems] = it;
            mbar_arrive(sh.bar + B_ITEM + k % kItems);
        }
        if (attn_withhold(p.a)) {
            ok = false;
            break;
        }
        if (more) ok = load_item(it);
    }
    // Whichever warp gives up, the copies in flight land before the CTA leaves (they have, if none did).
    if (lane == 0) {
        if (items > 0) mbar_wait_bounded(sh.bar + B_QFULL, (items - 1) & 1, kAttnWaitNs);
        for (int s = 0; s < kStages; ++s) {
            mbar_wait_bounded(sh.bar + B_KVFULL + s, ~(uses[0] >> s) & 1, kAttnWaitNs);
            mbar_wait_bounded(sh.bar + B_RAW + s, ~(uses[1] >> s) & 1, kAttnWaitNs);
        }
    }
}

// ---------------------------------------------------------------------------
// MMA
// ---------------------------------------------------------------------------
// Engine r's products, by one thread.  With two row tiles the engines take turns, a tile's p v and the next
// one's q k^T at a time, as in the windowed attention's kernel (the turn passes kPass MMAs into the latter).
constexpr int kPass = 5;
__device__ void mma_thread(const Params &p, Shared &sh, unsigned char *sm, int r) {
    const uint32_t tmem = sh.tmem;
    const uint64_t q0_desc = sw128_desc(smem_u32(sm + SM_Q)), q_desc = sw128_desc(smem_u32(sm + SM_Q + r * kTileBytes));
    const uint64_t k_desc = sw128_desc(smem_u32(sm + SM_KV)), v_desc = sw128_desc_mn(smem_u32(sm + SM_KV), kTileBytes / 2);
    constexpr uint64_t kTileStep = kTileBytes / 16;
    Ring ring;                                 // the next tile to be used
    uint32_t full_phase = 0, clean_phase = 0;  // bit s: phase of B_KVFULL, B_CLEAN + s
    uint32_t items = 0, p_phase = 0, turns = 0;
    bool ok = true;
    const auto full = [&](int stage) {
        const uint32_t phase = full_phase >> stage & 1;
        full_phase ^= 1u << stage;
        return wait_one(sh, B_KVFULL + stage, phase, p);
    };
    const auto clean = [&](int stage) {
        const uint32_t phase = clean_phase >> stage & 1;
        clean_phase ^= 1u << stage;
        return wait_one(sh, B_CLEAN + stage, phase, p);
    };
    // o += p v from the stage, in two halves as p comes
    const auto values = [&](int stage, bool first) {
        for (int half = 0; half < 2; ++half) {
            if (!wait_one(sh, B_P + 2 * r + half, p_phase, p)) return false;
            fence_after_sync();
            mma_values(tmem, v_desc + stage * kTileStep, r, half, first && half == 0);
        }
        p_phase ^= 1;
        return true;
    };
    const auto turn = [&] { return wait_one(sh, B_TURN + r, (turns++ + 1 + r) & 1, p); };  // engine 0 begins
    Items queue;
    while (ok) {
        const Item *at = queue.next<1>(sh, p);
        if (at == nullptr) break;
        const Item it = *at;
        queue.done(sh);
        const int32_t n = it.n;
        if (!(ok = wait_one(sh, B_QFULL, items & 1, p))) break;
        ++items;
        if (!it.two(p)) {
            // Every other tile.  The others are waited for and given back at once: a wait tells two neighbouring phases of a
            // barrier apart, so a place is not filled again before both engines have seen that it was.
            for (int32_t i = 0; i < n; ++i) {
                const int k = ring.stage;
                ring.next();
                const int v = ring.stage;
                ring.next();
                const bool tail = it.tail(i);
                if ((i & 1) != r) {
                    if (!(ok = full(k))) break;
                    mbar_arrive(sh.bar + B_KVEMPTY + k);
                    if (!(ok = tail ? clean(v) : full(v))) break;
                    mbar_arrive(sh.bar + B_KVEMPTY + v);
                    continue;
                }
                if (!(ok = full(k))) break;
                fence_after_sync();
                mma_scores(tmem, q0_desc, k_desc + k * kTileStep, r, 0, kD / 16);
                mma_commit(sh.bar + B_S + r);
                mma_commit(sh.bar + B_KVEMPTY + k);
                if (i + 2 >= n) mma_commit(sh.bar + B_QEMPTY);
                if (!(ok = tail ? clean(v) : full(v))) break;
                fence_after_sync();
                if (!(ok = values(v, i == r))) break;
                mma_commit(sh.bar + B_KVEMPTY + v);
                if (i + 2 >= n) mma_commit(sh.bar + B_O + r);
            }
            if (r >= n) mbar_arrive(sh.bar + B_QEMPTY);
            continue;
        }
        if (!(ok = full(ring.stage) && turn())) break;
        fence_after_sync();
        mma_scores(tmem, q_desc, k_desc + ring.stage * kTileStep, r, 0, kD / 16);
        mma_commit(sh.bar + B_S + r);
        mbar_arrive(sh.bar + B_TURN + 1 - r);
        mma_commit(sh.bar + B_KVEMPTY + ring.stage);
        if (n == 1) mma_commit(sh.bar + B_QEMPTY);
        ring.next();
        for (int32_t i = 0; i < n; ++i) {
            const int v = ring.stage;
            ring.next();
            const int k = ring.stage;
            const bool more = i + 1 < n;
            ok = it.tail(i) ? clean(v) : full(v);
            if (!ok || (more && !(ok = full(k)))) break;
            if (!(ok = turn() && values(v, i == 0))) break;
            if (!more) mma_commit(sh.bar + B_O + r);
            if (more) mma_scores(tmem, q_desc, k_desc + k * kTileStep, r, 0, kPass);
            mbar_arrive(sh.bar + B_TURN + 1 - r);
            if (more) {
                mma_scores(tmem, q_desc, k_desc + k * kTileStep, r, kPass, kD / 16);
                mma_commit(sh.bar + B_S + r);
            }
            mma_commit(sh.bar + B_KVEMPTY + v);
            if (more) {
                mma_commit(sh.bar + B_KVEMPTY + k);
                if (i + 2 == n) mma_commit(sh.bar + B_QEMPTY);
                ring.next();
            }
        }
    }
    // Whichever warp gives up, the MMAs in flight finish before TMEM is freed.
    mma_commit(sh.bar + B_DRAIN + r);
    mbar_wait_bounded(sh.bar + B_DRAIN + r, 0, kAttnWaitNs);
}

// ---------------------------------------------------------------------------
// Values behind the prefix's end
// ---------------------------------------------------------------------------
__device__ void clear_warp(const Params &p, Shared &sh, unsigned char *sm) {
    const int t = threadIdx.x & 31;
    Ring ring;
    uint32_t raw_phase = 0;  // bit s: phase of B_RAW + s
    Items queue;
    while (const Item *at = queue.next(sh, p)) {
        const Item it = *at;
        __syncwarp();
        if (t == 0) queue.done(sh);
        for (int32_t i = 0; i < it.n; ++i) {
            ring.next();  // k
            const Ring v = ring;
            ring.next();
            if (!it.tail(i)) continue;
            if (!wait(sh, B_RAW + v.stage, raw_phase >> v.stage & 1, p)) return;
            raw_phase ^= 1u << v.stage;
            // the rest of the group of 16 that the prefix ends in (the groups behind it were never fetched: zeros)
            unsigned char *tile = sm + SM_KV + v.stage * kTileBytes;
            const int32_t end = it.len - it.key(i), key = (end & ~15) + (t & 15);
            if (key >= end && key < kTile)
#pragma unroll
                for (int c = 0; c < 8; ++c)  // half of its 16-byte chunks, apart in the banks from lane to lane
                    *reinterpret_cast<uint4 *>(tile + (t >> 4) * (kTileBytes / 2) + 128 * key + 16 * ((c ^ key) & 7)) =
                        make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (t == 0) mbar_arrive(sh.bar + B_CLEAN + v.stage);
        }
    }
}

// ---------------------------------------------------------------------------
// Softmax and epilogue
// ---------------------------------------------------------------------------
// 16 channels of each lane's row to memory: four lanes (rows) exchange 16-byte chunks so that each store covers 64
// contiguous bytes of eight rows.  to[u]: the place of row 4 (lane / 4) + u, -1: none.
__device__ __forceinline__ void store16(const float (&o)[16], float *dst, const int32_t (&to)[4]) {
    const int lane = threadIdx.x & 31;
    uint32_t x[4][4];
#pragma unroll
    for (int u = 0; u < 16; ++u) x[u >> 2][u & 3] = __float_as_uint(o[u]);
#pragma unroll
    for (int bit = 2; bit > 0; bit >>= 1)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (!(u & bit)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool upper = lane & bit;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[u][k] : x[u ^ bit][k], bit);
                    if (upper) x[u][k] = got;
                    else x[u ^ bit][k] = got;
                }
            }
#pragma unroll
    for (int u = 0; u < 4; ++u)  // chunk lane % 4 of row 4 (lane / 4) + u
        if (to[u] >= 0)
            *reinterpret_cast<uint4 *>(dst + (int64_t)to[u] * kD + 4 * (lane & 3)) = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
}

__device__ void softmax_warps(const Params &p, Shared &sh, int r) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = 32 * quarter + lane;  // of the row tile
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_tmem = sh.tmem + lanes + 128 * r, o_tmem = sh.tmem + lanes + 256;
    uint32_t s_phase = 0, o_phase[2] = {0, 0}, join_phase = 0, tiles = 0;
    Items queue;
    while (const Item *it = queue.next<2>(sh, p)) {
        const int32_t n = it->n;
        const bool two = it->two(p);
        const int32_t tk = (int)((uint32_t)row * p.inv_g >> 16), token = (two ? r * p.tq : 0) + tk;
        const bool live = tk < p.tq && token < it->tokens;
        float m = -INFINITY, l = 0.f;
        const int32_t i0 = two ? 0 : r, step = two ? 1 : 2;
        for (int32_t i = i0; i < n; i += step) {
            if (!wait_inline(sh, B_S + r, s_phase, p)) return;
            s_phase ^= 1;
            fence_after_sync();
            uint32_t s[4][32];
            float top[4];
            tmem_ld32_async(s_tmem, s[0]);
            tmem_ld32_async(s_tmem + 32, s[1]);
            const uint32_t place = (tiles + i) % kTiles;
            const bool masked = *reinterpret_cast<const volatile uint32_t *>(sh.masked + place) != 0;
            tmem_ld_wait32(s[0]);
            tmem_ld_wait32(s[1]);
            tmem_ld32_async(s_tmem + 64, s[2]);
            tmem_ld32_async(s_tmem + 96, s[3]);
            if (!masked) {
                top[0] = max32(s[0]);
                top[1] = max32(s[1]);
            }
            tmem_ld_wait32(s[2]);
            tmem_ld_wait32(s[3]);
            if (masked) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t bits = reinterpret_cast<const volatile uint32_t *>(sh.mask + place)[c];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(bits >> k & 1)) s[c][k] = kMinusInf;
                }
                top[0] = max32(s[0]);
                top[1] = max32(s[1]);
            }
            top[2] = max32(s[2]);
            top[3] = max32(s[3]);
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            // lazily: only past 2^8 (from -inf at the row's first visible key)
            const bool move = (now - m) * p.c > 8.f && live;
            if (__any_sync(0xffffffffu, move)) {
                const float f = move ? ex2_approx((m - now) * p.c) : 1.f;
                if (move) m = now;
                l *= f;
                // s of this tile is complete, so the products issued before it are as well
                if (i > i0) {
#pragma unroll 1
                    for (int c = 0; c < 16; ++c) {
                        float o[8];
                        tmem_ld8(o_tmem + 128 * r + 8 * c, o);
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[k] * f);
                        tmem_st8u(o_tmem + 128 * r + 8 * c, u);
                    }
                    tmem_wait_st();
                }
            }
            const float base = m == -INFINITY ? 0.f : -m * p.c;
            const float2 c2 = make_float2(p.c, p.c), b2 = make_float2(base, base);
            float2 sum = make_float2(0.f, 0.f), sum2 = sum;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t out[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 x = fma2(make_float2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), c2, b2);
                    const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    if (k & 1) sum2 = add2(e, sum2);
                    else sum = add2(e, sum);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
                    out[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
                tmem_st16u(s_tmem + 16 * c, out);
                if (c & 1) {  // half of p is there: its products may start
                    tmem_wait_st();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.bar + B_P + 2 * r + (c >> 1));
                }
            }
            l += (sum.x + sum.y) + (sum2.x + sum2.y);
        }
        tiles += n;

        // The part's place, and each row's in it.
        const PrefixSpace space = prefix_space(p.a);
        const bool goes_on = it->goes_on;
        float *slot = prefix_slot(space, p.cut, (int32_t)blockIdx.x), *part = goes_on ? slot : space.o;
        const auto row_at = [&](int rt) {  // row rt of the row tile
            const int k = (int)((uint32_t)rt * p.inv_g >> 16), t = (two ? r * p.tq : 0) + k;
            if (k >= p.tq || t >= it->tokens) return -1;
            return goes_on ? (two ? r * kTile : 0) + rt : (it->first + t) * p.a.num_q_heads + it->h * p.cut.G + rt - k * p.cut.G;
        };
        int32_t to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) to[u] = row_at(32 * quarter + (lane & ~3) + u);
        const int32_t mine = row_at(row);
        float2 w = make_float2(m, l);
        if (two) {
            if (!wait_inline(sh, B_O + r, o_phase[r], p)) return;
            o_phase[0] ^= 1;
            o_phase[1] ^= 1;
        } else {
            // The engines' results joined: each half of the warps takes half of the channels.
            if (r == 1) {
                sh.ml[row] = w;
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.bar + B_JOIN);
                if (!wait_inline(sh, B_WEIGHTS, join_phase, p)) return;
                w = sh.ml[row];
            } else {
                if (!wait_inline(sh, B_JOIN, join_phase, p)) return;
                const float2 other = sh.ml[row];
                const float best = fmaxf(m, other.x);
                const auto weight = [&](float mx, float lx) {  // (a NaN sum stays one)
                    return mx == -INFINITY ? (lx == 0.f ? 0.f : 1.f) : ex2_approx((mx - best) * p.c);
                };
                w = make_float2(weight(m, l), weight(other.x, other.y));
                sh.ml[row] = w;
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.bar + B_WEIGHTS);
                l = w.x * l + w.y * other.y;
                m = best;
            }
            if (!wait_inline(sh, B_O, o_phase[0], p)) return;
            o_phase[0] ^= 1;
            if (n > 1) {
                if (!wait_inline(sh, B_O + 1, o_phase[1], p)) return;
                o_phase[1] ^= 1;
            }
        }
        fence_after_sync();
        const uint32_t from = o_tmem + (two ? 128 * r : 0);
        const bool both = !two && n > 1;
#pragma unroll 1
        for (int c = two ? 0 : 4 * r; c < (two ? 8 : 4 * r + 4); ++c) {
            float o[16];
            tmem_ld16(from + 16 * c, o);
            if (both) {
                float o1[16];
                tmem_ld16(from + 128 + 16 * c, o1);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = fmaf(w.y, o1[k], w.x * o[k]);
            }
            store16(o, part + 16 * c, to);
        }
        if (mine >= 0 && (two || r == 0)) {
            (goes_on ? prefix_slot_ml(slot, p.cut) : space.ml)[mine] = make_float2(m, l);
            const int32_t head = row - tk * p.cut.G;  // where the token's parts lie is said once for its query heads
            if (!goes_on && head == 0)
                space.more[(int64_t)(it->first + token) * p.a.num_kv_heads + it->h] =
                    make_int4((int32_t)blockIdx.x, it->more, sh.run.width, (two ? r * kTile : 0) + row);
        }
        fence_before_sync();  // the next item's products write o after this engine's next p
        __syncwarp();
        if (!two) {  // nor before the other half of the warps has read it
            if (lane == 0) mbar_arrive(sh.bar + B_JOINED);
            if (!wait_inline(sh, B_JOINED, join_phase, p)) return;
            join_phase ^= 1;
        }
        if (lane == 0) queue.done(sh);
    }
}

__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(const __grid_constant__ Params p) {
    extern __shared__ unsigned char dyn[];
    __shared__ Shared sh;
    unsigned char *sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(sh.bar + i, i == B_QEMPTY || (i >= B_KVEMPTY && i < B_CLEAN) ? 2
                                  : i >= B_P && i < B_O                             ? 4
                                  : i >= B_ITEMFREE && i < B_DRAIN                  ? kItemReaders
                                  : i == B_JOIN || i == B_WEIGHTS                   ? 4
                                  : i == B_JOINED                                   ? 8
                                                                                    : 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    grid_wait();
    prefix_begin(p.a, prefix_space(p.a));
    prefix_make_plan<kThreads>(p.a, p.cut, sh.run, sh.sums);  // (and __syncthreads)
    fence_after_sync();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_warps(p, sh, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kWarpTma) tma_warp(p, sh, sm);
        else if (warp == kWarpScrub) clear_warp(p, sh, sm);
        else if ((threadIdx.x & 31) == 0) mma_thread(p, sh, sm, warp - kWarpMma);
    }
    __syncthreads();
    if (warp == kWarpMma) tmem_dealloc(sh.tmem, 512);
    if (threadIdx.x == 0) prefix_space(p.a).done[blockIdx.x] = !sh.run.bad && sh.abort == 0;
}

}  // namespace

// How many neighbouring items of a group and kv head go side by side.  Each reads the same keys: where they do not fit
// into L2, items that go through them at different times fetch them from HBM again each, at 64 KB a CTA for
// the 1.1 us that a tile of 256 rows takes: 9.2 TB/s in all, 1.37 times what HBM gives.  Teams of two or more bring
// that below it, but leave CTAs over, and work for nothing where an item is missing in a team.
static int32_t team_width(const PrefixAttentionArgs &a, int32_t tokens, int32_t ctas) {
    const int64_t T = a.cache.total_tokens, items = ((T + a.num_groups - 1) / a.num_groups + tokens - 1) / tokens;
    const int64_t keys = (int64_t)a.cache.table_width * a.cache.page_size * a.num_groups;
    if (items == 1 || keys * a.num_kv_heads * (4 * kD) < (96ll << 20)) return 1;
    int32_t best = 1;
    double most = 1 / 1.37;
    for (int32_t w = 2; w <= 8; ++w) {
        const double share = (double)items / (double)((items + w - 1) / w * w) * (ctas / w * w) / ctas;
        if (share >= most) {
            most = share;
            best = w;
        }
    }
    return best;
}

PrefixCut prefix_cut_tc(const PrefixAttentionArgs &a, int32_t sms) {
    const int32_t G = a.num_q_heads / a.num_kv_heads, tq = kTile / G;
    return PrefixCut{0, G, 2 * tq, kTile, sms, 2 * kTile, a.num_groups > 0 ? team_width(a, 2 * tq, sms) : 1, 1.6f};
}

cudaError_t launch_prefix_tc(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream) {
    Params p;
    p.a = a;
    p.cut = cut;
    p.tq = cut.tile / 2;
    p.inv_g = (65536u + cut.G - 1) / cut.G;
    p.kv_rows = (int32_t)(2ll * a.cache.num_pages * a.num_kv_heads * a.cache.page_size);
    p.page_shift = a.cache.page_size == 16 ? 4 : a.cache.page_size == 32 ? 5 : a.cache.page_size == 64 ? 6 : 7;
    p.c = (float)((double)a.scale * 1.4426950408889634);
    if (!encode_kv_map(&p.tm_kv, a.kv_pool, a.cache, a.num_kv_heads, a.cache.page_size) ||
        !encode_kv_map(&p.tm_edge, a.kv_pool, a.cache, a.num_kv_heads, 16) ||
        !encode_q_map(&p.tm_q, a.q, a.cache.total_tokens, a.num_q_heads, cut.G, p.tq))
        return cudaErrorNotSupported;
    const cudaError_t e = allow_smem(prefix_tc_kernel, SM_DYN);
    return e == cudaSuccess ? launch_serial(prefix_tc_kernel, dim3((unsigned)cut.ctas), kThreads, SM_DYN, stream, p) : e;
}

}  // namespace kda
