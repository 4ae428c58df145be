// What the kernels of kda_prefix_attention share: the groups and requests of a step, how the work on the
// prefixes is shared out, and where partial results lie.
//
// Every row's (o, not divided; m; l) over the shared keys of its group and over its request's own keys are
// computed apart, the first for all requests of a group together, and joined in the last launch:
//   M = max m_i;  o = (sum_i e^(m_i - M) o_i) / (sum_i e^(m_i - M) l_i)
// The first launch goes over the prefixes, the second over the own keys (a CTA, or a cluster, a request and kv
// head).  They run side by side: the first leaves as many SMs to the second, which need not wait for it, as the
// work asks for, since they are bound by different things (tensor core and HBM).
//
// Prefixes: a work item is a tile of rows ((token, query head) pairs of one kv head, all requests of a group in
// one sequence) and the prefix.  The key tiles of all items, one after the other, are cut into runs of equal
// length, a run a CTA, wherever the cuts fall; an item spans as many CTAs as it needs, and counts
// kPrefixExtra tiles more than it has, for its beginning and end.  A part that starts an item is written to the
// rows' places in an array over all rows of the step; a part that goes on with an item that another CTA
// started (the first of a CTA's run, and only that) to the CTA's own slot.  `width` neighbouring items of a kv
// head may go side by side to as many CTAs (a team), so that their keys come from HBM once.
#pragma once

#include "kda_window_attention.cuh"

namespace kda {

// How rows and keys are cut: by rows (FMA kernels) an item has `tile` rows, else `tile` tokens.
struct PrefixCut {
    int32_t by_rows, G, tile;
    int32_t keys;       // of a tile
    int32_t ctas;       // of the first launch
    int32_t slot_rows;  // of a CTA's slot
    int32_t width;
    float tile_us;      // what a key tile takes a CTA
};
// In tiles.  With 2: 42 prompts x 60 beams 224 us instead of 215, 47 x 100 branches of few keys 1,115 instead of 970; no
// difference to long items.
constexpr int32_t kPrefixExtra = 3;
// What an own key of a kv head, and a request and kv head, take of an SM: 512 bytes at some 75 GB/s, and what their
// beginning and end cost, less where most keys are few (below 48 on average: heads go side by side).  They only say
// how SMs are shared out.  Too little for the own keys: 16 prompts x 4 beams 90 us with 0.7 instead of 79 with 2;
// too much: 256 requests behind a system prompt 253 us with 3, 236 with 2; 42 x 60 beams of 14 own keys 215 us
// with 2 for short ones too, 186 with 1.
constexpr float kOwnKeyUs = 512.f / 75e3f, kOwnItemUs = 2.f, kOwnShortUs = 1.f;

// Group g, checked; items = 0 when there is nothing to do for it (ok: whether it is well formed).
struct PrefixGroup {
    int32_t r0, r1, first, tokens, row, len;
    int32_t items, tiles;  // of a kv head
    bool ok;
};
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixAttentionArgs &a, const PrefixCut &cut, int32_t g) {
    const CacheArgs &c = a.cache;
    PrefixGroup x{a.cu_groups[g], a.cu_groups[g + 1], 0, 0, 0, 0, 0, 0, false};
    if (x.r0 < 0 || x.r1 <= x.r0 || x.r1 > c.batch) return x;
    x.first = c.cu_tokens[x.r0];
    const int32_t end = c.cu_tokens[x.r1];
    x.row = c.slot[x.r0];
    x.len = a.prefix_len[g];
    x.ok = x.first >= 0 && end >= x.first && end <= c.total_tokens && (uint32_t)x.row < (uint32_t)c.table_rows &&
           x.len >= 0 && x.len <= c.table_width * c.page_size;
    if (!x.ok) return x;
    x.tokens = end - x.first;
    x.tiles = (int32_t)(((uint32_t)x.len + cut.keys - 1) / cut.keys);
    if (x.tiles > 0) x.items = (int32_t)(((int64_t)x.tokens * (cut.by_rows ? cut.G : 1) + cut.tile - 1) / cut.tile);
    return x;
}

// Request b, checked: n = 0 when it is refused (then ok is false) or brings no tokens.
struct PrefixRequest {
    int32_t first, n, row, len;  // its tokens [first, first + n), its row, and the tokens in that
    int32_t from;                // its own keys start here
    bool ok;
};
__device__ __forceinline__ PrefixRequest prefix_request(const PrefixAttentionArgs &a, const PrefixCut &cut, int32_t b) {
    const CacheArgs &c = a.cache;
    int32_t lo = 0, hi = a.num_groups - 1;  // the last group that starts at or before b
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (a.cu_groups[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    const PrefixGroup x = prefix_group(a, cut, lo);
    PrefixRequest r{c.cu_tokens[b], 0, c.slot[b], 0, x.len, false};
    const int32_t end = c.cu_tokens[b + 1];
    if (!x.ok || b < x.r0 || b >= x.r1 || r.first < x.first || end < r.first || end - x.first > x.tokens ||
        end - r.first > a.max_tokens || (uint32_t)r.row >= (uint32_t)c.table_rows)
        return r;
    r.len = c.kv_len[r.row];
    r.ok = r.len >= 0 && r.len <= c.table_width * c.page_size && x.len <= r.len - (end - r.first);
    if (r.ok) r.n = end - r.first;
    return r;
}

// The workspace: a word a CTA of the first launch (1: it has done its run), and by rows of
// [T][Hq] the parts of prefixes (o [rows][128], (m, l) [rows]) and of own keys (o, (m, l, whether there is a
// prefix) with l < 0 where there is no result), for each token and kv head the CTAs that have parts of its rows'
// prefix, and the CTAs' slots (o, (m, l)).
constexpr int32_t kPrefixSms = 152;              // SMs that it is laid out for: the GPU's, but no more than these
constexpr int32_t kPrefixCtas = 2 * kPrefixSms;  // most CTAs of the first launch
struct PrefixSpace {
    uint32_t *done, *taken;  // taken: items of the second launch that a CTA has
    float *o, *own_o;
    float2 *ml;
    float4 *own;
    int4 *more;  // [T][Hkv] (by rows: [T][Hq]): (CTA, how many go on, from one to the next, the row in a slot of the
                 // kv head's first query head, or of the row)
    float *slots;
};
__host__ __device__ constexpr size_t prefix_round(size_t bytes) { return (bytes + 255) / 256 * 256; }
__host__ __device__ inline size_t prefix_space_at(const PrefixAttentionArgs &a, PrefixSpace *s) {
    unsigned char *w = static_cast<unsigned char *>(a.workspace);
    const size_t rows = (size_t)a.cache.total_tokens * a.num_q_heads;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        unsigned char *p = w + at;
        at += prefix_round(bytes);
        return p;
    };
    s->done = reinterpret_cast<uint32_t *>(take((kPrefixCtas + 1) * sizeof(uint32_t)));
    s->taken = s->done + kPrefixCtas;
    s->o = reinterpret_cast<float *>(take(rows * kD * sizeof(float)));
    s->own_o = reinterpret_cast<float *>(take(rows * kD * sizeof(float)));
    s->ml = reinterpret_cast<float2 *>(take(rows * sizeof(float2)));
    s->own = reinterpret_cast<float4 *>(take(rows * sizeof(float4)));
    s->more = reinterpret_cast<int4 *>(take(rows * sizeof(int4)));
    s->slots = reinterpret_cast<float *>(w + at);
    return at;
}
__device__ __forceinline__ PrefixSpace prefix_space(const PrefixAttentionArgs &a) {
    PrefixSpace s;
    prefix_space_at(a, &s);
    return s;
}
constexpr int64_t kSlotRow = kD + 2;  // floats
__device__ __forceinline__ float *prefix_slot(const PrefixSpace &s, const PrefixCut &cut, int32_t cta) {
    return s.slots + (int64_t)cta * cut.slot_rows * kSlotRow;
}
__device__ __forceinline__ float2 *prefix_slot_ml(float *slot, const PrefixCut &cut) {
    return reinterpret_cast<float2 *>(slot + cut.slot_rows * kD);
}

// At the beginning of the first launch, by all its threads: no row has a result.  Then what comes after may begin: the
// second launch, which writes the rows of its requests.  The barrier is what orders the two, since the first
// thread of a CTA that triggers speaks for all of it.
__device__ __forceinline__ void prefix_begin(const PrefixAttentionArgs &a, const PrefixSpace &s) {
    const int64_t rows = (int64_t)a.cache.total_tokens * a.num_q_heads;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows; i += (int64_t)gridDim.x * blockDim.x)
        s.own[i] = make_float4(0.f, -1.f, 0.f, 0.f);
    if (blockIdx.x == 0 && threadIdx.x == 0) *s.taken = 0;
    __threadfence();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// x / n for x >= 0 (64-bit divisions take some hundred cycles)
__device__ __forceinline__ int64_t prefix_div(int64_t x, int64_t n) {
    return (uint64_t)(x | n) <= 0xffffffffull ? (int64_t)((uint32_t)x / (uint32_t)n) : x / n;
}
// Team t of n takes units [units t / n, units (t + 1) / n) (n <= units); the team that has unit u:
__device__ __forceinline__ int64_t prefix_cut_at(int64_t units, int32_t t, int32_t n) { return prefix_div(units * t, n); }
__device__ __forceinline__ int32_t prefix_team(int64_t units, int64_t u, int32_t n) {
    return (int32_t)prefix_div((u + 1) * n + units - 1, units) - 1;
}

// The sum of x over the threads before this one; *all_x, *all_y: the sums over all.  All kThreads (a multiple of 32)
// call it; warp_sums: 2 kThreads / 32.
template <int kThreads>
__device__ __forceinline__ int64_t prefix_scan(int64_t x, int64_t y, int64_t *warp_sums, int64_t *all_x, int64_t *all_y) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, inc, off), t = __shfl_down_sync(0xffffffffu, y, off);
        if (lane >= off) inc += z;
        y += t;  // (lane 0: all)
    }
    if (lane == 31) warp_sums[warp] = inc;
    if (lane == 0) warp_sums[kWarps + warp] = y;
    __syncthreads();
    int64_t before = inc - x;
    *all_x = *all_y = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        *all_x += warp_sums[w];
        *all_y += warp_sums[kWarps + w];
    }
    return before;
}

// A CTA's run: units [from, to) of `all`, and the group that unit `from` lies in, with the units before it.
struct PrefixRun {
    int64_t from, to, all, units;
    int32_t team, teams, lane, width;
    int32_t at, bad;
    PrefixGroup x;
};

// Every CTA of the first launch works out the whole plan (a few loads a group and request).  `run` and `sums`
// (2 kThreads / 32) are in shared memory.
template <int kThreads>
__device__ void prefix_make_plan(const PrefixAttentionArgs &a, const PrefixCut &cut, PrefixRun &run, int64_t *sums) {
    const int32_t Ng = a.num_groups, B = a.cache.batch, Hkv = a.num_kv_heads, tid = threadIdx.x;
    const int32_t each = (Ng + kThreads - 1) / kThreads, g0 = min(tid * each, Ng), g1 = min(g0 + each, Ng);
    int64_t before = 0, own_keys = 0;  // (of the rows, less the prefixes)
    for (int32_t b = tid; b < B; b += kThreads) {
        const int32_t row = a.cache.slot[b];
        if ((uint32_t)row < (uint32_t)a.cache.table_rows) own_keys += a.cache.kv_len[row];
    }
    bool falls = false, mine = false;
    // first the work of this thread's groups is summed up, then the CTA's run finds its place among them
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int64_t units = 0;
        for (int32_t g = g0; g < g1; ++g) {
            const PrefixGroup x = prefix_group(a, cut, g);
            const int64_t n = (int64_t)Hkv * ((x.items + cut.width - 1) / cut.width) * (x.tiles + kPrefixExtra);
            if (x.r1 < x.r0) {
                falls = true;
                if (pass == 0 && blockIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)g);
            }
            if (x.ok) own_keys -= (int64_t)x.len * (x.r1 - x.r0);
            if (mine && run.from >= before + units && run.from < before + units + n) {
                run.at = g;
                run.units = before + units;
                run.x = x;
            }
            units += n;
        }
        if (pass == 1) break;
        int64_t all;
        before = prefix_scan<kThreads>(units, own_keys, sums, &all, &own_keys);
        falls = __syncthreads_or(falls);
        if (falls) all = 0;
        if (tid == 0) {
            // The own keys' launch gets the SMs that its work asks for, though never more than seven of eight: what is left
            // of it flows to SMs that the prefixes leave, the other way round it does not (1,210 branches of one own
            // key and 64 shared ones: 64 us, without 176).  Every team has a unit, so that the parts of an item
            // lie in neighbouring runs.
            const float work = (float)all * (float)cut.width * cut.tile_us;
            // (twice for more than 32 rows of a request, and so on)
            const float rows = (float)a.cache.total_tokens / (float)B * (float)(a.num_q_heads / Hkv);
            const float own_item = own_keys < 48ll * B ? kOwnShortUs : kOwnItemUs;
            const float own_work = (kOwnKeyUs * (float)max(own_keys, (int64_t)0) + own_item * (float)B) * (float)Hkv * fmaxf(1.f, rows / 32.f);
            int32_t teams = (int32_t)((float)cut.ctas * work / (work + own_work) / (float)cut.width + 0.5f);
            teams = max(cut.ctas / (8 * cut.width), min(teams, cut.ctas / cut.width));
            // And where a CTA would have less than four units, fewer do, down to a third: the others are free for the own
            // keys at once, and there are fewer parts to join (those 10 beams: 26 us instead of 33; six prompts of one
            // request 23 instead of 29).
            teams = (int32_t)min((int64_t)teams, max(all / 4, min(all, (int64_t)(cut.ctas / 3))));
            run.teams = teams = max(teams, (int32_t)min(all, (int64_t)1));  // (a GPU of few SMs)
            run.all = all;
            run.width = cut.width;
            run.bad = falls;
            run.team = (int32_t)blockIdx.x / cut.width;
            run.lane = (int32_t)blockIdx.x % cut.width;
            run.from = run.team < teams ? prefix_cut_at(all, run.team, teams) : 0;
            run.to = run.team < teams ? prefix_cut_at(all, run.team + 1, teams) : 0;
        }
        __syncthreads();
        mine = run.from < run.to;
        if (!mine) break;  // (the whole CTA)
    }
    __syncthreads();
}

// One stretch of a CTA's run: key tiles [tile, tile + count) of one item.
struct PrefixStretch {
    int32_t first, tokens, row, len;  // of the group
    int32_t h, index, items;          // kv head; number of the row tile and how many there are
    int32_t tile, count;
    bool goes_on;                     // with an item that another CTA started: the part goes to the CTA's slot
    int32_t more;                     // else: CTAs that go on with it
};

// Walks the stretches of a run, item after item by counting.  Every thread that calls it gets the same answers.
struct PrefixWalk {
    int64_t u, units;
    int32_t at;                     // the group at hand, from unit `units` on
    int32_t inside = 0, item = -1;  // unit of its item `item`; -1: not begun
    int32_t per, items, wide;       // units of an item, items of all kv heads and of one
    int32_t h, index;
    PrefixGroup x;

    __device__ __forceinline__ explicit PrefixWalk(const PrefixRun &run) : u(run.from), units(run.units), at(run.at) {}
    __device__ __forceinline__ bool next(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run,
                                         PrefixStretch &s) {
        while (u < run.to) {
            if (item < 0 && !begin(a, cut, run)) {
                u = run.to;  // (never: u < run.to <= all units)
                return false;
            }
            const int32_t end = (int32_t)min((int64_t)per, inside + (run.to - u));
            s.first = x.first; s.tokens = x.tokens; s.row = x.row; s.len = x.len; s.items = x.items;
            s.h = h;
            s.index = index * run.width + run.lane;
            s.goes_on = inside > kPrefixExtra;
            s.tile = max(0, inside - kPrefixExtra);
            s.count = end - kPrefixExtra - s.tile;
            s.more = end == per ? 0 : prefix_team(run.all, u - inside + per - 1, run.teams) - run.team;
            u += end - inside;
            inside = 0;
            if (++index == wide) {
                index = 0;
                ++h;
            }
            if (++item == items) {
                item = -1;
                units += (int64_t)items * per;
                ++at;
            }
            if (s.count > 0 && s.index < s.items) return true;
        }
        return false;
    }

  private:
    __device__ __forceinline__ bool begin(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run) {
        for (; at < a.num_groups; ++at) {
            x = run.x;
            if (at != run.at) x = prefix_group(a, cut, at);
            wide = (x.items + run.width - 1) / run.width;
            per = x.tiles + kPrefixExtra;
            items = a.num_kv_heads * wide;
            if (u < units + (int64_t)items * per) {
                item = (int32_t)prefix_div(u - units, per);
                inside = (int32_t)(u - units - (int64_t)item * per);
                h = item / wide;
                index = item - h * wide;
                return true;
            }
            units += (int64_t)items * per;
        }
        return false;
    }
};

// For a GPU of `sms` SMs (at most kPrefixSms): with fewer CTAs than these the first launch would leave some idle, with more its
// last ones would begin when the others are done, and with them all of the second launch.
PrefixCut prefix_cut_rows(const PrefixAttentionArgs &a, int32_t sms);
PrefixCut prefix_cut_tc(const PrefixAttentionArgs &a, int32_t sms);
cudaError_t launch_prefix_tc(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);
cudaError_t launch_prefix_own(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);

}  // namespace kda
