// Sliding-window attention over the paged cache on the tensor cores (bf16): prefill, chunked
// prefill, and any step whose requests bring more rows than the split-row kernel takes.
//
//   s = q k^T;  p = 2^(c s - c m), c = scale log2 e;  l += sum p;  o += p v;  at the end o / l
// The reference m of a row follows its running maximum lazily: it moves (and o, l are scaled by
// 2^(c (m_old - m_new))) only when a score exceeds it by more than 2^8 in p, so that p <= 2^8 and
// almost every tile leaves o alone; the division by l removes the choice of m again.  s, m, l and
// o are fp32; p enters its product rounded to bf16 (the tensor core takes both operands in one
// type), which costs at most 2^-8 of each weight.
//
// A work item is 2 x 128 rows of one request and key/value head; a row is a (token, query head of
// the group) pair, so that the heads of a group share every key and value, and a tile of 128 rows
// spans only 128 / G tokens: the window's edges then cost few masked tiles.  Keys come in tiles of
// 128, those of the sinks first.  The grid has a CTA an item; one an SM starts and, when done with its
// item, takes over one that has not started (cluster launch control), so that SMs that are slower at the
// moment take fewer.  With few items a cluster of up to eight CTAs shares the key tiles of one, and joins
// the partial results through distributed shared memory (in an order that the sizes alone decide).
//   warp 8      TMA: q of the next item, then k, v tiles page by page into a ring of five 32 KB
//               stages (a page that does not exist is an out-of-range box, which reads as zeros)
//   warps 9, 10 issue the MMAs of row tiles 0 and 1: s = q k^T into TMEM, o += p v with p read from
//               TMEM (in place of s).  While one row tile's softmax runs, the tensor core works on
//               the other's products
//   warps 0-7   softmax, a thread a row: warps 0-3 tile 0, warps 4-7 tile 1; the epilogue
//   warp 11     values behind a mask: a product with p = 0 would still turn NaN or infinity into
//               NaN, so tiles that some row must not see are gone through first: keys that no row
//               sees are cleared, and a non-finite value of any other key marks the item, whose
//               rows are at the end computed again one by one, each from its visible keys alone.
// TMEM: s0, s1, o0, o1 of 128 columns each.  Bound: the tensor core (two 128 x 128 x 128 products
// a key tile and row tile, 512 cycles each at its full rate).
// Measured: 2 x 16,384 tokens behind cached ones, window 4096 + 16, 32 query and 8 kv heads: 1.49 ms,
// 1310 TFLOP/s (0.70 of a large bf16 GEMM's rate; 1.42 in bursts of a few launches, before the power limit
// tells); 8192 tokens, window 1024 + 4, 96 and 8 heads: 0.52 to 0.575 ms from run to run, for no cause that was
// found (0.45 at best), 0.74 to 0.68 PFLOP/s: of its ten key tiles an item four are on an edge, which costs a softmax
// warp about 1,700 cycles more.  Scores read from TMEM twice instead of held: 3.17 ms on the first; four
// stages instead of five: 5 % slower; work in fixed turns: 1.44 ms (where these were 1.42) and up to 0.60.
// Two issuing warps over two row tiles, and a maximum that moves only past 2^8, are published methods for
// attention on this chip.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_window_attention.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kTile = 128;                    // rows of a row tile, keys of a key tile
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr int kStages = 5;
constexpr int kItems = 4;                     // work items announced ahead
constexpr int kPitchO = kD + 4;               // floats of a row's partial result: o, m, l
constexpr int kTainted = 200;                 // marked items a CTA keeps; it takes no more work near the end
constexpr int kItemReaders = 11;              // warps that read them: softmax, MMA, values
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpScrub = 11;
// 384 threads start with 168 registers; the softmax warps take 208, the others keep 88:
// 256 * 208 + 128 * 88 = 384 * 168
constexpr int kRegsSoftmax = 208, kRegsOther = 88;

enum Bar {
    B_QFULL, B_QEMPTY, B_KVFULL, B_RAW = B_KVFULL + kStages, B_KVEMPTY = B_RAW + kStages,
    B_CLEAN = B_KVEMPTY + kStages,
    B_S = B_CLEAN + kStages, B_P = B_S + 2, B_O = B_P + 4, B_ITEM = B_O + 2, B_ITEMFREE = B_ITEM + kItems,
    B_DRAIN = B_ITEMFREE + kItems, B_TURN = B_DRAIN + 2, B_NEXT = B_TURN + 2, B_COUNT
};

constexpr uint32_t SM_Q = 0, SM_KV = 2 * kTileBytes, SM_END = SM_KV + kStages * kTileBytes;
constexpr size_t SM_DYN = SM_END + 1024;  // the start is rounded up to 1024 bytes

struct Params {
    CUtensorMap tm_q;   // [T][Hq][128], boxes of tq tokens x G heads x 64 channels
    CUtensorMap tm_kv;  // [2 P Hkv page_size][128], boxes of a page x 64 channels
    WindowAttentionArgs a;
    int32_t G, tq;      // query heads a kv head, tokens of a row tile
    uint32_t inv_g;     // ceil(2^16 / G): x / G = x inv_g >> 16 for x < 128
    int32_t kv_rows;    // 2 P Hkv page_size
    int32_t page_shift;  // log2 page_size
    float c;            // scale log2 e, > 0
};

// (a.x + b.x, a.y + b.y)
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    return fma2(a, make_float2(1.f, 1.f), b);
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// One work item, found by the TMA warp and left in shared memory for the others.
struct Item {
    int32_t first, tokens;     // its tokens: rows [first, first + tokens) of q and o
    int32_t h, row;            // kv head, row of the table
    int32_t p_min, p_max;      // indices of its first and last token
    int32_t n;                 // key tiles; < 0: no more items
    int32_t from;              // the first of its tiles among those of the keys its tokens see
    int32_t sink_tiles, skip;  // of those, tile i starts at key 128 (i < sink_tiles ? i : i + skip)

    __device__ __forceinline__ int32_t key(int32_t i) const {
        return kTile * (from + i < sink_tiles ? from + i : from + i + skip);
    }
    __device__ __forceinline__ bool two(const Params &p) const { return tokens > p.tq; }  // a second row tile
    // Some row of the item must not see some key of the tile that starts at j0.
    __device__ __forceinline__ bool masked(int32_t j0, const Params &p) const {
        return masked(j0, p_min, p_max, p);
    }
    static __device__ __forceinline__ bool masked(int32_t j0, int32_t lo, int32_t hi, const Params &p) {
        return j0 + (kTile - 1) > lo || (hi - j0 >= p.a.window && j0 + (kTile - 1) >= p.a.sinks);
    }
};

struct Shared {
    uint64_t bar[B_COUNT];
    Item items[kItems];
    int2 tiles[8];  // by key tile % 8: its first key; bit i: its page i exists, bit 16 + r: some row of row tile r
                    // must not see some key of it
    uint4 next;                  // the answer to the load warp's request for more work
    uint32_t work[kItems];       // numbers of the items in `items`
    uint32_t tainted[kTainted];  // numbers of the items whose masked tiles held a non-finite value
    uint32_t tainted_count;
    uint32_t tmem;
    uint32_t abort;
};

// One thread waits for a phase, giving up after attn_wait_ns() or when another warp has given up.
__device__ __forceinline__ bool wait_one(Shared &sh, int bar, uint32_t parity, const Params &p) {
    if (mbar_try_wait(sh.bar + bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (mbar_try_wait(sh.bar + bar, parity)) return true;
        if (attn_given_up(&sh.abort)) return false;
        if (global_timer_ns() - t0 > attn_wait_ns(p.a)) {
            attn_give_up(&sh.abort, p.a, (uint32_t)(64 + bar));
            return false;
        }
    }
}
// A warp does, all lanes to one verdict.
__device__ __forceinline__ bool wait(Shared &sh, int bar, uint32_t parity, const Params &p) {
    return attn_wait_warp(sh.bar + bar, parity, &sh.abort, p.a, (uint32_t)(64 + bar));
}

// The ring of k, v stages: tile loads in order, stage n % kStages, phase n / kStages.  A load
// completes B_KVFULL of its stage, or B_RAW when the tile is values to be gone through first
// (B_CLEAN follows); those barriers' phases are counted by use, a bit a stage.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The items in turn, for the warps that read them.
struct Items {
    uint32_t k = 0;
    // The next item, in its place until done(); null after the last one or when a wait gave up.  A whole
    // warp calls it, or (kOne) one thread for its warp.
    template <bool kOne = false>
    __device__ __forceinline__ const Item *next(Shared &sh, const Params &p) {
        const uint32_t slot = k % kItems;
        const bool there = kOne ? wait_one(sh, B_ITEM + slot, k / kItems & 1, p) : wait(sh, B_ITEM + slot, k / kItems & 1, p);
        if (!there) return nullptr;
        ++k;
        return sh.items[slot].n >= 0 ? &sh.items[slot] : nullptr;
    }
    // By one thread of the warp, which has read all it wants.
    __device__ __forceinline__ void done(Shared &sh) { mbar_arrive(sh.bar + B_ITEMFREE + (k - 1) % kItems); }
};

// ---------------------------------------------------------------------------
// TMA
// ---------------------------------------------------------------------------
// Work item w, or n = -1 past the last one.
__device__ __forceinline__ Item find_item(const Params &p, AttnWalk &walk, int64_t w, AttnRequest &req) {
    const int32_t Hkv = p.a.num_kv_heads, tokens = 2 * p.tq;
    Item it;
    int32_t index;
    it.n = -1;
    if (w / Hkv < walk.before) walk = AttnWalk();  // work comes in order, as a rule
    if (!walk.find(p.a, w / Hkv, 1, tokens, req, index)) return it;
    // the last tokens of a request first: with little out of the window they see most keys
    const int32_t t0 = ((req.n + tokens - 1) / tokens - 1 - index) * tokens;
    it.first = req.first + t0;
    it.tokens = min(tokens, req.n - t0);
    it.h = (int32_t)(w % Hkv);
    it.row = req.row;
    it.p_min = req.len - req.n + t0;
    it.p_max = it.p_min + it.tokens - 1;
    const AttnKeys keys(it.p_min, it.p_max, p.a.window, p.a.sinks, kTile);
    it.n = keys.count();
    it.from = 0;
    it.sink_tiles = keys.sink_tiles;
    it.skip = keys.low_tile - keys.sink_tiles;
    return it;
}

// Cluster launch control: asks the scheduler to withdraw a CTA of this grid that has not started.  The
// answer comes to shared memory: whether there was one, and which.
__device__ __forceinline__ void request_work(uint4 *answer, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool taken_work(const uint4 *answer, uint32_t &w) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}\n"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    if (ok) w = x;
    return ok != 0;
}

template <bool kSplit>
__device__ void tma_warp(const Params &p, Shared &sh, unsigned char *sm) {
    const int lane = threadIdx.x & 31;
    const int32_t page = p.a.cache.page_size, pages = kTile / page;  // pages of a tile
    const uint32_t all_pages = (1u << pages) - 1u;
    Ring ring;
    uint32_t loads = 0, items = 0, tiles = 0, uses[2] = {0, 0};  // bit s: parity of the uses of KVFULL, RAW + s
    bool ok = true;
    uint32_t asked = 0;  // requests for more work that were answered
    bool asking = false;  // one is under way
    // The grid has a CTA an item: those that have not started are taken over, one at a time.
    const auto ask = [&] {
        if (kSplit) return;
        const uint32_t marked = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(&sh.tainted_count), 0);
        asking = marked + 2 * kItems < kTainted;
        if (asking && lane == 0) {
            fence_proxy_async_smem();  // the last answer has been read
            mbar_arrive_expect_tx(sh.bar + B_NEXT, 16);
            request_work(&sh.next, sh.bar + B_NEXT);
        }
    };
    // q, k and v of one item
    const auto load_item = [&](const Item &it) {
        const bool two = it.two(p);
        const auto load_q = [&] {  // when the last item's scores are done
            if (items > 0 && !wait(sh, B_QEMPTY, (items - 1) & 1, p)) return false;
            ++items;
            if (lane != 0) return true;
            const uint32_t bytes = (uint32_t)(p.tq * p.G * 64 * 2);
            mbar_arrive_expect_tx(sh.bar + B_QFULL, bytes * (two ? 4u : 2u));
            for (int r = 0; r < (two ? 2 : 1); ++r)
                for (int half = 0; half < 2; ++half)
                    tma_load_3d(smem_u32(sm + SM_Q + r * kTileBytes + half * (kTileBytes / 2)), &p.tm_q,
                                64 * half, it.h * p.G, it.first + r * p.tq, sh.bar + B_QFULL);
            return true;
        };
        for (int32_t i = 0; ok && i < it.n; ++i) {
            const int32_t j0 = it.key(i);
            // lane = 2 page + half: that page's rows of the tile, 64 channels
            int32_t id = -1;
            if (lane < 2 * pages) id = attn_page(p.a.cache, it.row, it.p_max, j0 / page + (lane >> 1));
            const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
            for (int kv = 0; kv < 2; ++kv) {
                if (loads >= kStages && !(ok = wait(sh, B_KVEMPTY + ring.stage, ring.phase ^ 1, p))) break;
                const int raw = kv == 1 && it.masked(j0, p) ? 1 : 0;
                uint64_t *full = sh.bar + (raw ? B_RAW : B_KVFULL) + ring.stage;
                uses[raw] ^= 1u << ring.stage;
                if (lane == 0) {
                    if (kv == 0) {  // at most three tiles are ahead of a softmax: eight places do
                        uint32_t bits = 0;
                        for (int32_t u = 0; u < pages; ++u) bits |= (exist >> (2 * u) & 1) << u;
                        for (int32_t r = 0; r < 2; ++r) {
                            const int32_t lo = it.p_min + r * p.tq, hi = min(lo + p.tq - 1, it.p_max);
                            if (bits != all_pages || Item::masked(j0, lo, hi, p)) bits |= 0x10000u << r;
                        }
                        sh.tiles[tiles & 7] = make_int2(j0, (int)bits);
                    }
                    mbar_arrive_expect_tx(full, kTileBytes);
                }
                __syncwarp();
                if (lane < 2 * pages) {
                    const int32_t y = id < 0 ? p.kv_rows  // out of range: zeros
                                             : ((id * 2 + kv) * p.a.num_kv_heads + it.h) * page;
                    tma_load_2d(smem_u32(sm + SM_KV + ring.stage * kTileBytes + (lane & 1) * (kTileBytes / 2) +
                                         (lane >> 1) * page * 128),
                                &p.tm_kv, 64 * (lane & 1), y, full);
                }
                ring.next();
                ++loads;
                if (i == 0 && kv == 0 && !(ok = load_q())) break;  // q behind the first keys
            }
            ++tiles;
            if (ok && i == 0) ask();  // behind the first loads
        }
        return ok;
    };
    AttnWalk walk;
    AttnRequest req;
    uint32_t w = kSplit ? blockIdx.x / cluster_size() : blockIdx.x;
    bool more = true;
    for (uint32_t k = 0; ok && more;) {
        Item it = find_item(p, walk, w, req);
        if (kSplit && it.n > 0) {  // this CTA's share of the item's tiles
            const int32_t rank = (int32_t)cluster_rank(), size = (int32_t)cluster_size(), n = it.n;
            it.from = (int32_t)((int64_t)n * rank / size);
            it.n = (int32_t)((int64_t)n * (rank + 1) / size) - it.from;
        }
        if (it.n >= 0) {
            if (k >= kItems && !(ok = wait(sh, B_ITEMFREE + k % kItems, (k / kItems - 1) & 1, p))) break;
            if (lane == 0) {
                sh.items[k % kItems] = it;
                sh.work[k % kItems] = w;
                mbar_arrive(sh.bar + B_ITEM + k % kItems);
            }
            ++k;
        }
        if (attn_withhold(p.a)) {
            ok = false;
            break;
        }
        if (it.n <= 0) ask();
        else if (!(ok = load_item(it))) break;
        if (asking) {
            if (!(ok = wait(sh, B_NEXT, asked & 1, p))) break;
            ++asked;
            asking = false;
            more = taken_work(&sh.next, w);
            __syncwarp();
        } else {
            more = false;
        }
        if (!more) {
            if (k >= kItems && !(ok = wait(sh, B_ITEMFREE + k % kItems, (k / kItems - 1) & 1, p))) break;
            if (lane == 0) {
                sh.items[k % kItems].n = -1;
                mbar_arrive(sh.bar + B_ITEM + k % kItems);
            }
        }
    }
    // Whichever warp gives up, the copies in flight land before the CTA leaves (they have, if none did).
    if (lane == 0) {
        if (items > 0) mbar_wait_bounded(sh.bar + B_QFULL, (items - 1) & 1, kAttnWaitNs);
        if (asking) mbar_wait_bounded(sh.bar + B_NEXT, asked & 1, kAttnWaitNs);
        for (int s = 0; s < kStages; ++s) {
            mbar_wait_bounded(sh.bar + B_KVFULL + s, ~(uses[0] >> s) & 1, kAttnWaitNs);
            mbar_wait_bounded(sh.bar + B_RAW + s, ~(uses[1] >> s) & 1, kAttnWaitNs);
        }
    }
}

// ---------------------------------------------------------------------------
// MMA
// ---------------------------------------------------------------------------
// One 128-wide product is eight MMAs of 64 cycles each, all issued by one thread: their matrix
// descriptors differ from the first one's by constants (16-byte units of the address field).
__device__ __forceinline__ void mma_scores(uint32_t tmem, uint64_t q_desc, uint64_t k_desc, int r, int from, int to) {
#pragma unroll
    for (int s = from; s < to; ++s) {
        const uint64_t step = ((s >> 2) * (kTileBytes / 2) + (s & 3) * 32) / 16;
        mma_bf16(tmem + 128 * r, q_desc + step, k_desc + step, idesc_bf16_f32(kTile, kTile), s > 0);
    }
}
// Keys 64 half .. 64 half + 63 of a tile.
__device__ __forceinline__ void mma_values(uint32_t tmem, uint64_t v_desc, int r, int half, bool first) {
#pragma unroll
    for (int s = 4 * half; s < 4 * half + 4; ++s)
        mma_bf16_tmem_a(tmem + 256 + 128 * r, tmem + 128 * r + 8 * s, v_desc + s * (2048 / 16),
                        idesc_bf16_f32(kTile, kD) | kIdescBMN, s > 0 ? 1u : !first);
}

// Row tile r's products, by one thread.  The tensor core runs them as they are issued, so what a
// thread does between two products (waits, bookkeeping) is hidden by the other row tile's thread.
// The two take turns, a tile's p v and the next one's q k^T at a time: left to interleave, both
// row tiles would wait for their products at once (2.03 ms for the 2 x 16384-token chunk at window
// 4096, against 1.52).  The turn passes kPass MMAs into the second product, about the 250 cycles
// ahead that the other thread takes to see it (all 8 done: 1.63 ms, none: 1.65).
constexpr int kPass = 5;
__device__ void mma_thread(const Params &p, Shared &sh, unsigned char *sm, int r) {
    const uint32_t tmem = sh.tmem;
    const uint64_t q_desc = sw128_desc(smem_u32(sm + SM_Q + r * kTileBytes));
    const uint64_t k_desc = sw128_desc(smem_u32(sm + SM_KV)), v_desc = sw128_desc_mn(smem_u32(sm + SM_KV), kTileBytes / 2);
    constexpr uint64_t kTileStep = kTileBytes / 16;
    Ring ring;                                 // the next tile to be used
    uint32_t full_phase = 0, clean_phase = 0;  // bit s: phase of B_KVFULL, B_CLEAN + s
    uint32_t items = 0, p_phase = 0;
    bool ok = true;
    // frees what both threads use: by this one's products, or at once when it has none
    const auto release = [&](int bar, bool two) {
        if (r == 0 || two) mma_commit(sh.bar + bar);
        else mbar_arrive(sh.bar + bar);
    };
    const auto full = [&](int stage) {
        const uint32_t phase = full_phase >> stage & 1;
        full_phase ^= 1u << stage;
        return wait_one(sh, B_KVFULL + stage, phase, p);
    };
    uint32_t turns = 0;
    const auto turn = [&] { return wait_one(sh, B_TURN + r, (turns++ + 1 + r) & 1, p); };  // row tile 0 begins
    Items queue;
    while (ok) {
        const Item *at = queue.next<true>(sh, p);
        if (at == nullptr) break;
        const Item it = *at;
        queue.done(sh);
        const int32_t n = it.n;
        const bool two = it.two(p), mine = r == 0 || two;
        if (n == 0) continue;
        if (!(ok = wait_one(sh, B_QFULL, items & 1, p) && full(ring.stage))) break;
        ++items;
        fence_after_sync();
        if (mine) {
            if (two && !(ok = turn())) break;
            mma_scores(tmem, q_desc, k_desc + ring.stage * kTileStep, r, 0, kD / 16);
            mma_commit(sh.bar + B_S + r);
            if (two) mbar_arrive(sh.bar + B_TURN + 1 - r);
        }
        release(B_KVEMPTY + ring.stage, two);
        if (n == 1) release(B_QEMPTY, two);
        ring.next();
        for (int32_t i = 0; i < n; ++i) {
            const int v = ring.stage;
            ring.next();
            const int k = ring.stage;
            const bool more = i + 1 < n;
            if (it.masked(it.key(i), p)) {
                ok = wait_one(sh, B_CLEAN + v, clean_phase >> v & 1, p);
                clean_phase ^= 1u << v;
            } else {
                ok = full(v);
            }
            if (!ok || (more && !(ok = full(k)))) break;
            if (mine) {
                if (two && !(ok = turn())) break;
                if (!(ok = wait_one(sh, B_P + 2 * r, p_phase, p))) break;
                fence_after_sync();
                mma_values(tmem, v_desc + v * kTileStep, r, 0, i == 0);
                if (!(ok = wait_one(sh, B_P + 2 * r + 1, p_phase, p))) break;
                p_phase ^= 1;
                fence_after_sync();
                mma_values(tmem, v_desc + v * kTileStep, r, 1, false);
                if (!more) mma_commit(sh.bar + B_O + r);
                if (more) mma_scores(tmem, q_desc, k_desc + k * kTileStep, r, 0, kPass);
                if (two) mbar_arrive(sh.bar + B_TURN + 1 - r);
                if (more) {
                    mma_scores(tmem, q_desc, k_desc + k * kTileStep, r, kPass, kD / 16);
                    mma_commit(sh.bar + B_S + r);
                }
            }
            release(B_KVEMPTY + v, two);
            if (more) {
                release(B_KVEMPTY + k, two);
                if (i + 2 == n) release(B_QEMPTY, two);
                ring.next();
            }
        }
    }
    // Whichever warp gives up, the MMAs in flight finish before TMEM is freed.
    mma_commit(sh.bar + B_DRAIN + r);
    mbar_wait_bounded(sh.bar + B_DRAIN + r, 0, kAttnWaitNs);
}

// ---------------------------------------------------------------------------
// Values behind a mask
// ---------------------------------------------------------------------------
__device__ void scrub_warp(const Params &p, Shared &sh, unsigned char *sm) {
    const int t = threadIdx.x & 31;
    Ring ring;
    uint32_t raw_phase = 0;  // bit s: phase of B_RAW + s
    Items queue;
    while (const Item *at = queue.next(sh, p)) {
        const Item it = *at;
        const uint32_t work = sh.work[(queue.k - 1) % kItems];
        __syncwarp();
        if (t == 0) queue.done(sh);
        bool marked = false;
        for (int32_t i = 0; i < it.n; ++i) {
            ring.next();  // k
            const Ring v = ring;
            ring.next();
            const int32_t j0 = it.key(i);
            if (!it.masked(j0, p)) continue;
            if (!wait(sh, B_RAW + v.stage, raw_phase >> v.stage & 1, p)) return;
            raw_phase ^= 1u << v.stage;
            unsigned char *tile = sm + SM_KV + v.stage * kTileBytes;
            uint32_t bad = 0;
#pragma unroll 1
            for (int key = t; key < kTile; key += 32) {
                const int32_t j = j0 + key;
                const bool sink = j < p.a.sinks;
                if (j <= it.p_min && (sink || it.p_max - j < p.a.window)) continue;  // every row sees it
                // some row sees it: not past the last token, and within the first token's reach
                const bool seen = j <= it.p_max && (sink || it.p_min - j < p.a.window);
#pragma unroll
                for (int c = 0; c < 16; ++c) {  // its 16-byte chunks, apart in the banks from lane to lane
                    uint4 *x = reinterpret_cast<uint4 *>(tile + (c >> 3) * (kTileBytes / 2) + 128 * key +
                                                         16 * ((c ^ key) & 7));
                    if (seen) {
                        const uint4 y = *x;
                        bad |= any_nonfinite(y.x) | any_nonfinite(y.y) | any_nonfinite(y.z) | any_nonfinite(y.w);
                    } else {
                        *x = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            __syncwarp();
            marked |= __any_sync(0xffffffffu, bad != 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (t == 0) mbar_arrive(sh.bar + B_CLEAN + v.stage);
        }
        if (marked && t == 0 && sh.tainted_count < kTainted) {  // (always: no work is taken near the end)
            sh.tainted[sh.tainted_count] = work;
            *reinterpret_cast<volatile uint32_t *>(&sh.tainted_count) = sh.tainted_count + 1;
        }
    }
}

// ---------------------------------------------------------------------------
// Softmax and epilogue
// ---------------------------------------------------------------------------
constexpr uint32_t kMinusInf = 0xff800000u;

// The lowest n bits (none for n < 0, all from 32 on).
__device__ __forceinline__ uint32_t low_mask(int32_t n) {
    uint32_t m;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(max(n, 0)));
    return m;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
    float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
    for (int k = 2; k < 30; k += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
        b = fmaxf(fmaxf(b, __uint_as_float(s[k + 2])), __uint_as_float(s[k + 3]));
    }
    return fmaxf(fmaxf(a, b), fmaxf(__uint_as_float(s[30]), __uint_as_float(s[31])));
}

// A split item's partial results of one row: o as it is, then m and l.
__device__ __forceinline__ float *partial_row(unsigned char *sm, int r, int row) {
    return reinterpret_cast<float *>(sm + SM_KV) + (kTile * r + row) * kPitchO;
}
__device__ __forceinline__ void keep_partial(uint32_t o_tmem, bool any, float m, float l, float *dst) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float o[32];
        if (any) tmem_ld32(o_tmem + 32 * c, o);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4 *>(dst + 32 * c + k) =
                any ? make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    *reinterpret_cast<float2 *>(dst + kD) = make_float2(m, l);
}

// Writes a row tile's outputs.  Four lanes (rows) exchange 16-byte chunks so that each store covers
// 64 contiguous bytes of eight rows; a row a thread, the 32 lines of every store kept the load/store
// unit busy for 4,000 cycles an item.
__device__ __forceinline__ void store_rows(const Params &p, uint32_t o_tmem, bool any, float l, __nv_bfloat16 *o_item,
                                           int32_t token0, int32_t tokens) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *out = o_item + 8 * (lane & 3);
    int32_t to[4];  // rows 4 (lane / 4) + u of the tile, as rows of [T][Hq] from the item's first; -1: none
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int rt = 32 * quarter + (lane & ~3) + u;
        const int tk = (int)((uint32_t)rt * p.inv_g >> 16), tt = token0 + tk;
        to[u] = tk < p.tq && tt < tokens ? tt * p.a.num_q_heads + rt - tk * p.G : -1;
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {  // 32 channels: chunks 0 .. 3
        uint32_t x[4][4];
        {
            uint32_t o[32];
            if (any) {
                tmem_ld32_async(o_tmem + 32 * c, o);
                tmem_ld_wait32(o);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const __nv_bfloat162 h =
                    __floats2bfloat162_rn(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
                // no key: 0, whatever o holds (a NaN sum stays one)
                x[u >> 2][u & 3] = l == 0.f ? 0u : *reinterpret_cast<const uint32_t *>(&h);
            }
        }
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
                *reinterpret_cast<uint4 *>(out + (int64_t)to[u] * kD + 32 * c) =
                    make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
    }
}

template <bool kSplit>
__device__ void softmax_warps(const Params &p, Shared &sh, unsigned char *sm, int r) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = 32 * quarter + lane;  // of the row tile
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_tmem = sh.tmem + lanes + 128 * r, o_tmem = sh.tmem + lanes + 256 + 128 * r;
    const WindowAttentionArgs &a = p.a;
    // this row: its token of the item and query head (rows from tq G on are empty)
    const int32_t token = r * p.tq + row / p.G;
    uint32_t s_phase = 0, o_phase = 0, tiles = 0;
    Items queue;
    while (const Item *it = queue.next(sh, p)) {
        const int32_t n = it->n;
        if (r == 1 && !it->two(p)) {
            tiles += n;
            __syncwarp();
            if (lane == 0) queue.done(sh);
            continue;
        }
        // the row's index (-1 sees nothing)
        const int32_t pos = row < p.tq * p.G && token < it->tokens ? it->p_min + token : -1;
        float m = -INFINITY, l = 0.f;
        for (int32_t i = 0; i < n; ++i, ++tiles) {
            if (!wait(sh, B_S + r, s_phase, p)) return;
            s_phase ^= 1;
            fence_after_sync();
            uint32_t s[4][32];
            float top[4];
            tmem_ld32_async(s_tmem, s[0]);
            tmem_ld32_async(s_tmem + 32, s[1]);
            const uint32_t mapped = *reinterpret_cast<volatile uint32_t *>(&sh.tiles[tiles & 7].y);
            const bool masked = mapped & 0x10000u << r;
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
                const int32_t j0 = *reinterpret_cast<volatile int32_t *>(&sh.tiles[tiles & 7].x);
                const int32_t hi = pos - j0 + 1, lo = pos < a.window ? 0 : pos - a.window + 1 - j0;
                const int32_t sk = a.sinks - j0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t bits = low_mask(hi - 32 * c) & (~low_mask(lo - 32 * c) | low_mask(sk - 32 * c));
                    if (p.page_shift == 4) bits &= (mapped >> (2 * c) & 1 ? 0xffffu : 0u) | (mapped >> (2 * c + 1) & 1 ? 0xffff0000u : 0u);
                    else if (!(mapped >> (32 * c >> p.page_shift) & 1)) bits = 0;
                    // most 32-key chunks of an edge tile need nothing (a way out for unseen ones too spilled)
                    if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(bits >> k & 1)) s[c][k] = kMinusInf;
                }
            }
            if (masked) {
                top[0] = max32(s[0]);
                top[1] = max32(s[1]);
            }
            top[2] = max32(s[2]);
            top[3] = max32(s[3]);
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            // lazily: only past 2^8 (from -inf at the row's first visible key)
            const bool move = (now - m) * p.c > 8.f;
            if (__any_sync(0xffffffffu, move)) {
                const float f = move ? ex2_approx((m - now) * p.c) : 1.f;
                if (move) m = now;
                l *= f;
                // s of this tile is complete, so the products issued before it are as well
                if (i > 0) {
#pragma unroll 1
                    for (int c = 0; c < 16; ++c) {
                        float o[8];
                        tmem_ld8(o_tmem + 8 * c, o);
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[k] * f);
                        tmem_st8u(o_tmem + 8 * c, u);
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

        if (n > 0) {
            if (!wait(sh, B_O + r, o_phase, p)) return;
            // the partial results will lie where the other row tile's values do
            if (kSplit && it->two(p) && !wait(sh, B_O + 1 - r, o_phase, p)) return;
            o_phase ^= 1;
            fence_after_sync();
        }
        if (kSplit) {
            keep_partial(o_tmem, n > 0, m, l, partial_row(sm, r, row));
            if (lane == 0) queue.done(sh);
            continue;
        }
        store_rows(p, o_tmem, n > 0, l, static_cast<__nv_bfloat16 *>(a.o) + ((int64_t)it->first * a.num_q_heads + it->h * p.G) * kD,
                   r * p.tq, it->tokens);
        if (lane == 0) queue.done(sh);
        fence_before_sync();  // the next item's products write o after this row tile's next p
    }
}

// The rows of this CTA's marked items again, by all warps.
__device__ __noinline__ void redo_tainted(const Params &p, const Shared &sh, int warp) {
    AttnWalk walk;
    AttnRequest req;
    for (uint32_t k = 0; k < sh.tainted_count; ++k) {
        const Item it = find_item(p, walk, sh.tainted[k], req);
        for (int32_t row = warp; row < it.tokens * p.G; row += kThreads / 32) {
            const int32_t token = row / p.G;
            attn_row(p.a, (int64_t)(it.first + token) * p.a.num_q_heads + it.h * p.G + row % p.G, it.h, it.row,
                     it.p_min + token);
        }
    }
}

// Joins a split item: its rows go round the cluster's warps, four channels a lane.
__device__ __noinline__ void join_split(const Params &p, Shared &sh, unsigned char *sm, int warp) {
    const int lane = threadIdx.x & 31;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    AttnWalk walk;
    AttnRequest req;
    const Item it = find_item(p, walk, blockIdx.x / size, req);
    if (it.n < 0) return;  // the whole cluster
    uint32_t failed = 0, tainted = 0;
    if (lane < (int)size) {
        failed = remote_u32(remote(smem_u32(&sh.abort), lane));
        tainted = remote_u32(remote(smem_u32(&sh.tainted_count), lane));
    }
    if (__any_sync(0xffffffffu, failed != 0)) return;
    tainted = __any_sync(0xffffffffu, tainted != 0);
    for (int32_t row = rank * (kThreads / 32) + warp; row < it.tokens * p.G; row += size * (kThreads / 32)) {
        const int32_t token = row / p.G, g = row - token * p.G;
        const int64_t q_row = (int64_t)(it.first + token) * p.a.num_q_heads + it.h * p.G + g;
        if (tainted) {
            attn_row(p.a, q_row, it.h, it.row, it.p_min + token);
            continue;
        }
        const int r = token >= p.tq ? 1 : 0;
        const uint32_t mine = smem_u32(partial_row(sm, r, (token - r * p.tq) * p.G + g));
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < (int)size) ml = remote_float2(remote(mine + kD * 4, lane));
        float top = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx((ml.x - top) * p.c);  // (a NaN sum stays one)
        float sum = w * ml.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t s = 0; s < size; ++s) {
            const float ws = __shfl_sync(0xffffffffu, w, s);
            const float4 x = remote_float4(remote(mine + 16 * lane, s));
            acc = make_float4(fmaf(ws, x.x, acc.x), fmaf(ws, x.y, acc.y), fmaf(ws, x.z, acc.z), fmaf(ws, x.w, acc.w));
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4(static_cast<__nv_bfloat16 *>(p.a.o) + q_row * kD + 4 * lane,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) attention_tc_kernel(const __grid_constant__ Params p) {
    extern __shared__ unsigned char dyn[];
    __shared__ Shared sh;
    unsigned char *sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(sh.bar + i, i == B_QEMPTY || (i >= B_KVEMPTY && i < B_CLEAN) ? 2
                                  : i >= B_P && i < B_O                             ? 4
                                  : i >= B_ITEMFREE && i < B_DRAIN                  ? kItemReaders
                                                                                    : 1);
        sh.abort = 0;
        sh.tainted_count = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    grid_wait();
    __syncthreads();
    fence_after_sync();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_warps<kSplit>(p, sh, sm, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kWarpTma) tma_warp<kSplit>(p, sh, sm);
        else if (warp == kWarpScrub) scrub_warp(p, sh, sm);
        else if ((threadIdx.x & 31) == 0) mma_thread(p, sh, sm, warp - kWarpMma);
    }
    __syncthreads();
    if (warp == kWarpMma) tmem_dealloc(sh.tmem, 512);
    if constexpr (kSplit) {
        cluster_sync();
        join_split(p, sh, sm, warp);
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its partials
    } else {
        if (sh.tainted_count != 0) redo_tainted(p, sh, warp);  // after every store of the first pass
    }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        return nullptr;
    }();
    return fn;
}

}  // namespace

bool encode_kv_map(CUtensorMap *m, const WindowAttentionArgs &a, int32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const CacheArgs &c = a.cache;
    const cuuint64_t dims[2] = {kD, 2ull * c.num_pages * a.num_kv_heads * c.page_size};
    const cuuint64_t strides[1] = {kD * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(a.kv_pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_kv_box_map(CUtensorMap *m, const WindowAttentionArgs &a, int32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const CacheArgs &c = a.cache;
    const cuuint64_t dims[4] = {64, 2ull * c.num_pages * a.num_kv_heads * c.page_size, 2, 2};
    const cuuint64_t strides[3] = {kD * 2, 128, (cuuint64_t)a.num_kv_heads * c.page_size * kD * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 2, 2}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(a.kv_pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_window_attention_tc(const WindowAttentionArgs &a, cudaStream_t stream) {
    Params p;
    p.a = a;
    p.G = a.num_q_heads / a.num_kv_heads;
    p.tq = kTile / p.G;
    p.inv_g = (65536u + p.G - 1) / p.G;
    p.kv_rows = (int32_t)(2ll * a.cache.num_pages * a.num_kv_heads * a.cache.page_size);
    p.page_shift = a.cache.page_size == 16 ? 4 : a.cache.page_size == 32 ? 5 : a.cache.page_size == 64 ? 6 : 7;
    p.c = (float)((double)a.scale * 1.4426950408889634);
    auto fn = tensor_map_encoder();
    if (fn == nullptr || !encode_kv_map(&p.tm_kv, a, a.cache.page_size)) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {kD, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.cache.total_tokens};
    const cuuint64_t strides[2] = {kD * 2, (cuuint64_t)a.num_q_heads * kD * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.tq}, estr[3] = {1, 1, 1};
    if (fn(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorNotSupported;
    // sum of ceil(n_b / tokens) over the requests, at most
    const int64_t tokens = 2 * p.tq;
    const int64_t items = (a.cache.total_tokens + a.cache.batch * (tokens - 1)) / tokens * a.num_kv_heads;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // Few items: a cluster shares each one's key tiles, as long as all CTAs are resident at once (a
    // cluster of 4 or 8 does not fill every group of SMs) and keep two tiles or more.
    const int64_t reach = (int64_t)a.window + tokens - 1 + a.sinks;
    const int64_t held = (int64_t)a.cache.table_width * a.cache.page_size;
    const int64_t tiles = ((reach < held ? reach : held) + kTile - 1) / kTile;
    const int64_t sms = device_sm_count();
    int splits = 1;
    while (splits < 8 && items * splits * 2 <= sms - (splits == 1 ? 0 : sms / 5) && tiles >= 4 * splits) splits *= 2;
    if (splits == 1) {
        const cudaError_t e = allow_smem(attention_tc_kernel<false>, SM_DYN);
        return e == cudaSuccess ? launch_serial(attention_tc_kernel<false>, dim3((unsigned)items), kThreads, SM_DYN, stream, p)
                                : e;
    }
    return launch_clusters(attention_tc_kernel<true>, dim3((unsigned)(items * splits)), splits, kThreads, SM_DYN, stream, p);
}

}  // namespace kda
