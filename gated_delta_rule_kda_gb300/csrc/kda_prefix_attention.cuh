// What the kernels of kda_prefix_attention share: the groups of a step, how the work on their prefixes
// is shared out, and where its partial results lie.
//
// The first launch goes over the prefixes, the second over each request's own keys, joins the two parts
// and writes o.  In the first, a work item is a tile of rows ((token, query head) pairs of one group and
// kv head, all requests of the group in one sequence) and a unit one item's tile of keys; the units of all
// items, one after the other, are cut into equal runs, a run a CTA, wherever the cuts fall (equal work
// whatever the lengths; an item spans as many CTAs as it needs).  `width` neighbouring items of a kv head
// go side by side as one, to as many CTAs (a team), so that their keys are fetched from HBM once.  A CTA
// leaves o (not divided), m and l of each stretch of an item in a slot of the workspace: slot
// (item + team) width + lane, which no other stretch has, since along the runs item and team never fall and
// one of them rises from stretch to stretch.
#pragma once

#include "kda_window_attention.cuh"

namespace kda {

// How rows and keys are cut.
struct PrefixCut {
    int32_t per, tile;  // a group of n tokens has ceil(n per / tile) items
    int32_t keys;       // of a tile
    int32_t ctas;       // of the first launch
    int32_t slots;      // of the workspace
};

// The head of the workspace.
struct PrefixPlan {
    int64_t units;   // of all groups; < 0: groups overlap, so that their items would not fit
    int32_t width, teams;
};
struct PrefixBase {
    int64_t units;   // before a group
    int32_t items;   // (of `width` row tiles) before it
    int32_t pad;
};

// Group g, checked; items = 0 when there is nothing to do for it (ok: whether it is well formed).
struct PrefixGroup {
    int32_t first, tokens, row, len;
    int32_t items, tiles;  // of a kv head
    bool ok;
};
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixAttentionArgs &a, const PrefixCut &cut, int32_t g) {
    const CacheArgs &c = a.cache;
    PrefixGroup x{0, 0, 0, 0, 0, 0, false};
    const int32_t r0 = a.cu_groups[g], r1 = a.cu_groups[g + 1];
    if (r0 < 0 || r1 <= r0 || r1 > c.batch) return x;
    x.first = c.cu_tokens[r0];
    const int32_t end = c.cu_tokens[r1];
    x.row = c.slot[r0];
    x.len = a.prefix_len[g];
    x.ok = x.first >= 0 && end >= x.first && end <= c.total_tokens && (uint32_t)x.row < (uint32_t)c.table_rows &&
           x.len >= 0 && x.len <= c.table_width * c.page_size;
    if (!x.ok) return x;
    x.tokens = end - x.first;
    x.tiles = (int32_t)(((uint32_t)x.len + cut.keys - 1) / cut.keys);
    x.items = (int32_t)(((int64_t)x.tokens * cut.per + cut.tile - 1) / cut.tile);
    if (x.tiles == 0) x.items = 0;
    return x;
}

// The workspace: plan, a word a CTA of the first launch (1: it has done its run), a base a group, then the slots.
constexpr int32_t kPrefixCtas = 2 * 152;  // most of them
__host__ __device__ inline size_t prefix_slots_at(int32_t num_groups) {
    return (sizeof(PrefixPlan) + kPrefixCtas * sizeof(uint32_t) + (size_t)num_groups * sizeof(PrefixBase) + 255) / 256 * 256;
}
__device__ __forceinline__ const PrefixPlan *prefix_plan(const PrefixAttentionArgs &a) {
    return static_cast<const PrefixPlan *>(a.workspace);
}
__device__ __forceinline__ uint32_t *prefix_done(const PrefixAttentionArgs &a) {
    return reinterpret_cast<uint32_t *>(static_cast<PrefixPlan *>(a.workspace) + 1);
}
__device__ __forceinline__ const PrefixBase *prefix_bases(const PrefixAttentionArgs &a) {
    return reinterpret_cast<const PrefixBase *>(prefix_done(a) + kPrefixCtas);
}
// A slot of `rows` rows: o as [rows][128], then (m, l) as [rows][2].
__host__ __device__ constexpr int64_t prefix_slot_floats(int32_t rows) { return (int64_t)rows * (kD + 2); }
__device__ __forceinline__ float *prefix_slot(const PrefixAttentionArgs &a, int32_t rows, int64_t slot) {
    return reinterpret_cast<float *>(static_cast<unsigned char *>(a.workspace) + prefix_slots_at(a.num_groups)) +
           slot * prefix_slot_floats(rows);
}

// Team t of n takes units [units t / n, units (t + 1) / n); the team that has unit u:
__device__ __forceinline__ int64_t prefix_cut(int64_t units, int32_t t, int32_t n) { return units * t / n; }
__device__ __forceinline__ int32_t prefix_team(int64_t units, int64_t u, int32_t n) {
    return (int32_t)(((u + 1) * n + units - 1) / units) - 1;
}

// Sum of x over the threads before this one; *total: over all.  All kThreads (a multiple of 32) call it.
template <int kThreads>
__device__ __forceinline__ int64_t prefix_scan(int64_t x, int64_t *warp_sums, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    __syncthreads();  // the last use of warp_sums is over
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + inc - x;
}

// A CTA's run of units, and the group it starts in.
struct PrefixRun {
    int64_t from, to;     // units
    int32_t group;        // that of unit `from` (from < to)
    int32_t team, lane;   // of the CTA
    int32_t width;
    PrefixBase base;      // of that group
};

// Every CTA of the first launch works out the whole plan (a few loads a group); CTA 0 writes it down.
// `run` and `sums` (kThreads / 32) are in shared memory.
template <int kThreads>
__device__ void prefix_make_plan(const PrefixAttentionArgs &a, const PrefixCut &cut, PrefixRun &run, int64_t *sums) {
    const int32_t Ng = a.num_groups, Hkv = a.num_kv_heads;
    const int32_t each = (Ng + kThreads - 1) / kThreads, g0 = threadIdx.x * each, g1 = min(g0 + each, Ng);
    const int32_t width = 1;
    int64_t units = 0, items = 0;
    for (int32_t g = g0; g < g1; ++g) {
        const PrefixGroup x = prefix_group(a, cut, g);
        items += (int64_t)Hkv * x.items;
        units += (int64_t)Hkv * x.items * x.tiles;
    }
    int64_t all_units, all_items;
    int64_t units_before = prefix_scan<kThreads>(units, sums, &all_units);
    int64_t items_before = prefix_scan<kThreads>(items, sums, &all_items);
    // every team has a unit: the parts of an item lie in one run of teams
    const int32_t teams = (int32_t)max((int64_t)1, min((int64_t)(cut.ctas / width), all_units));
    const bool fits = (all_items + teams) * width <= cut.slots;
    if (!fits) all_units = 0;
    if (threadIdx.x == 0) {
        run.team = (int32_t)blockIdx.x / width;
        run.lane = (int32_t)blockIdx.x % width;
        run.width = width;
        run.from = run.team < teams ? prefix_cut(all_units, run.team, teams) : 0;
        run.to = run.team < teams ? prefix_cut(all_units, run.team + 1, teams) : 0;
        if (blockIdx.x == 0) *static_cast<PrefixPlan *>(a.workspace) = PrefixPlan{fits ? all_units : -1, width, teams};
    }
    __syncthreads();
    for (int32_t g = g0; g < g1; ++g) {
        const PrefixGroup x = prefix_group(a, cut, g);
        const PrefixBase base{units_before, fits ? (int32_t)items_before : 0, 0};
        const int64_t n = (int64_t)Hkv * x.items * x.tiles;
        if (run.from < run.to && run.from >= units_before && run.from < units_before + n) {
            run.group = g;
            run.base = base;
        }
        if (blockIdx.x == 0) const_cast<PrefixBase *>(prefix_bases(a))[g] = base;
        units_before += n;
        items_before += (int64_t)Hkv * x.items;
    }
    __syncthreads();
}

// One stretch of a CTA's run: key tiles [tile, tile + count) of one item.
struct PrefixStretch {
    int32_t first, tokens, row, len;  // of the group
    int32_t h, index;                 // kv head; number of the row tile (at or past the last: nothing to do)
    int32_t items;                    // row tiles of the group
    int32_t tile, count;
    int64_t slot;
};
// Walks the stretches of a run; every thread that calls it gets the same answers.
struct PrefixWalk {
    int64_t u;
    int32_t g;
    PrefixBase base;
    PrefixGroup x;
    __device__ __forceinline__ PrefixWalk(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run)
        : u(run.from), g(run.group), base(run.base) {
        if (run.from < run.to) x = prefix_group(a, cut, g);
    }
    __device__ __forceinline__ bool next(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run,
                                         PrefixStretch &s) {
        if (u >= run.to) return false;
        const int32_t Hkv = a.num_kv_heads;
        int32_t wide = (x.items + run.width - 1) / run.width;  // items of a kv head, `width` row tiles each
        while (u >= base.units + (int64_t)Hkv * wide * x.tiles) {  // (ends: u < run.to <= all units)
            base.units += (int64_t)Hkv * wide * x.tiles;
            base.items += Hkv * wide;
            x = prefix_group(a, cut, ++g);
            wide = (x.items + run.width - 1) / run.width;
        }
        const int64_t at = u - base.units;
        const int32_t item = (int32_t)(at / x.tiles);
        s.tile = (int32_t)(at - (int64_t)item * x.tiles);
        s.count = (int32_t)min((int64_t)(x.tiles - s.tile), run.to - u);
        s.first = x.first; s.tokens = x.tokens; s.row = x.row; s.len = x.len;
        s.items = x.items;
        s.h = item / wide;
        s.index = (item - s.h * wide) * run.width + run.lane;
        s.slot = ((int64_t)base.items + item + run.team) * run.width + run.lane;
        u += s.count;
        return true;
    }
};

// The second launch's view: the slots that hold the partial results of row tile `index` of kv head h.
struct PrefixSlots {
    int64_t first;           // the first slot
    int32_t count, step;     // of them, and from one to the next
    int32_t cta;             // of the first; each slot's CTA is `step` after the one before
};
__device__ __forceinline__ PrefixSlots prefix_slots(const PrefixPlan &plan, const PrefixBase &base, const PrefixGroup &x,
                                                    int32_t h, int32_t index) {
    if (x.items == 0) return PrefixSlots{0, 0, 0, 0};
    const int32_t wide = (x.items + plan.width - 1) / plan.width, item = h * wide + index / plan.width;
    const int64_t u = base.units + (int64_t)item * x.tiles;
    const int32_t t0 = prefix_team(plan.units, u, plan.teams), t1 = prefix_team(plan.units, u + x.tiles - 1, plan.teams);
    return PrefixSlots{((int64_t)base.items + item + t0) * plan.width + index % plan.width, t1 - t0 + 1, plan.width,
                       t0 * plan.width + index % plan.width};
}

// Request b of the second launch, checked against its group; n = 0 when it is refused (then *bad).
struct PrefixRequest {
    AttnRequest req;
    PrefixGroup x;
    int32_t g;
};
__device__ __forceinline__ PrefixRequest prefix_request(const PrefixAttentionArgs &a, const PrefixCut &cut, int32_t b, bool *bad) {
    PrefixRequest r;
    const CacheArgs &c = a.cache;
    r.req = AttnRequest{b, c.cu_tokens[b], 0, c.slot[b], 0};
    int32_t lo = 0, hi = a.num_groups - 1;  // the last group that starts at or before b
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (a.cu_groups[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    r.g = lo;
    r.x = prefix_group(a, cut, lo);
    const int32_t end = c.cu_tokens[b + 1];
    bool ok = r.x.ok && a.cu_groups[lo] <= b && b < a.cu_groups[lo + 1] && r.req.first >= r.x.first &&
              end >= r.req.first && end - r.x.first <= r.x.tokens && end - r.req.first <= a.max_tokens &&
              (uint32_t)r.req.row < (uint32_t)c.table_rows;
    if (ok) {
        r.req.len = c.kv_len[r.req.row];
        ok = r.req.len >= 0 && r.req.len <= c.table_width * c.page_size && r.x.len <= r.req.len - (end - r.req.first);
    }
    if (ok) r.req.n = end - r.req.first;
    *bad = !ok;
    return r;
}

constexpr int32_t kPrefixTcRows = 256;  // of a slot of the tensor-core kernel: two row tiles
cudaError_t launch_prefix_tc(const PrefixAttentionArgs &a, cudaStream_t stream);
PrefixCut prefix_cut_tc(int32_t total_tokens, int32_t num_groups, int32_t num_q_heads, int32_t num_kv_heads);
cudaError_t launch_prefix_own(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);
PrefixCut prefix_cut_rows(int32_t total_tokens, int32_t num_groups, int32_t num_q_heads, int32_t num_kv_heads);
cudaError_t launch_prefix_rows(const PrefixAttentionArgs &a, cudaStream_t stream);

}  // namespace kda
