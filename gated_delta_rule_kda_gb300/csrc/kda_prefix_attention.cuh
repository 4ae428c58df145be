// What the kernels of kda_prefix_attention share: the groups and requests of a step, how their work is
// shared out, and where its partial results lie.
//
// Every row's (o, not divided; m; l) over the shared keys of its group and over its request's own keys are
// computed apart, the first for all requests of a group together, and joined in the last launch:
//   M = max m_i;  o = (sum_i e^(m_i - M) o_i) / (sum_i e^(m_i - M) l_i)
// A work item is a tile of rows ((token, query head) pairs of one kv head) with the keys they share: rows of
// all requests of a group and its prefix, or rows of one request and its own keys.  The key tiles of all items
// of a kind, one after the other, are cut into runs of equal length, a run a CTA, wherever the cuts fall; an
// item spans as many CTAs as it needs, and counts a few tiles more than it has, for its beginning and end.
//   fp32  one launch for both kinds: some CTAs take prefixes, the others own keys, in the ratio of the work
//   bf16  two launches: prefixes on the tensor cores (tcgen05), own keys on the warp-wide tensor
//         instruction, a cluster of CTAs a request and kv head.  They run side by side: the first leaves as
//         many SMs to the second, which need not wait for it, as the work asks for, since they are bound by
//         different things (tensor core and HBM)
// A part that starts an item is written to the rows' places in an array over all rows of the step (one array
// for prefixes, one for own keys); a part that goes on with an item that another CTA started (the first of
// a CTA's run, and only that) to the CTA's own slot.  `width` neighbouring items of a group and kv
// head may go side by side to as many CTAs (a team), so that their keys come from HBM once.
#pragma once

#include "kda_window_attention.cuh"

namespace kda {

// How rows and keys are cut: by rows (fp32 kernel) an item has `tile` rows, else `tile` tokens (prefixes) or
// `own_tile` tokens.
struct PrefixCut {
    int32_t by_rows, G, tile, own_tile;
    int32_t keys;       // of a tile
    int32_t ctas;       // of the first launch
    int32_t slot_rows;  // of a CTA's slot
    int32_t width;
    int32_t own_apart;  // own keys are another launch's
};
constexpr int32_t kPrefixExtra = 2, kOwnExtra = 1;

__host__ __device__ __forceinline__ int32_t prefix_items(const PrefixCut &c, int32_t tokens, int32_t tile) {
    return (int32_t)(((int64_t)tokens * (c.by_rows ? c.G : 1) + tile - 1) / tile);
}

// The head of the workspace.
struct PrefixPlan {
    int64_t units, own_units;  // tiles of all items of a kind
    int32_t bad;               // cu_groups falls somewhere: nothing is computed
    int32_t width, teams, own_ctas;  // CTAs [0, teams width) take prefixes, the next own_ctas own keys
};

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
    x.items = x.tiles == 0 ? 0 : prefix_items(cut, x.tokens, cut.tile);
    return x;
}

// The last group that starts at or before request b.
__device__ __forceinline__ int32_t prefix_group_of(const PrefixAttentionArgs &a, int32_t b) {
    int32_t lo = 0, hi = a.num_groups - 1;
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (a.cu_groups[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Request b of group x, checked: n = 0 when it is refused (then ok is false) or brings no tokens.
struct PrefixRequest {
    int32_t first, n, row, len;  // its tokens [first, first + n), its row, and the tokens in that
    int32_t from;                // its own keys start here
    int32_t items, tiles;        // of a kv head
    bool ok;
};
__device__ __forceinline__ PrefixRequest prefix_request(const PrefixAttentionArgs &a, const PrefixCut &cut,
                                                        const PrefixGroup &x, int32_t b) {
    const CacheArgs &c = a.cache;
    PrefixRequest r{c.cu_tokens[b], 0, c.slot[b], 0, x.len, 0, 0, false};
    const int32_t end = c.cu_tokens[b + 1];
    if (!x.ok || b < x.r0 || b >= x.r1 || r.first < x.first || end < r.first || end - x.first > x.tokens ||
        end - r.first > a.max_tokens || (uint32_t)r.row >= (uint32_t)c.table_rows)
        return r;
    r.len = c.kv_len[r.row];
    r.ok = r.len >= 0 && r.len <= c.table_width * c.page_size && x.len <= r.len - (end - r.first);
    if (!r.ok) return r;
    r.n = end - r.first;
    if (r.n == 0) return r;
    r.items = prefix_items(cut, r.n, cut.own_tile);
    r.tiles = (r.len - 1) / cut.keys - r.from / cut.keys + 1;  // (from <= len - n < len)
    return r;
}

// The workspace: plan, a word a CTA of the first launch (1: it has done its run), the units before each group
// and before each request, the rows' parts ([rows][128], then (m, l) as [rows][2]) of prefixes and of own
// keys, the CTAs' slots (alike).
constexpr int32_t kPrefixCtas = 2 * 152;  // most of them
struct PrefixSpace {
    int64_t *units, *own_units;  // [Ng], [B]
    uint32_t *done;
    float *part[2], *slots;
    int64_t rows;
};
__host__ __device__ inline size_t prefix_parts_at(int32_t num_groups, int32_t batch) {
    return (sizeof(PrefixPlan) + kPrefixCtas * sizeof(uint32_t) + ((size_t)num_groups + batch) * 8 + 255) / 256 * 256;
}
__host__ __device__ constexpr int64_t prefix_part_floats(int64_t rows) { return (rows * (kD + 2) + 63) / 64 * 64; }  // (16-byte vectors)
__device__ __forceinline__ PrefixSpace prefix_space(const PrefixAttentionArgs &a) {
    unsigned char *w = static_cast<unsigned char *>(a.workspace);
    PrefixSpace s;
    s.done = reinterpret_cast<uint32_t *>(w + sizeof(PrefixPlan));
    s.units = reinterpret_cast<int64_t *>(s.done + kPrefixCtas);
    s.own_units = s.units + a.num_groups;
    s.rows = (int64_t)a.cache.total_tokens * a.num_q_heads;
    s.part[0] = reinterpret_cast<float *>(w + prefix_parts_at(a.num_groups, a.cache.batch));
    s.part[1] = s.part[0] + prefix_part_floats(s.rows);
    s.slots = s.part[1] + prefix_part_floats(s.rows);
    return s;
}
// Rows of a part: o at row 128, (m, l) behind all rows.
struct PrefixPart {
    float *o;
    float2 *ml;
};
__device__ __forceinline__ PrefixPart prefix_part(const PrefixSpace &s, int own) {
    return PrefixPart{s.part[own], reinterpret_cast<float2 *>(s.part[own] + s.rows * kD)};
}
__device__ __forceinline__ PrefixPart prefix_slot(const PrefixSpace &s, const PrefixCut &cut, int32_t cta) {
    float *o = s.slots + (int64_t)cta * cut.slot_rows * (kD + 2);
    return PrefixPart{o, reinterpret_cast<float2 *>(o + cut.slot_rows * kD)};
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

// A CTA's run: units [from, to) of its kind, and the group or request that unit `from` lies in.
struct PrefixRun {
    int64_t from, to, units;  // units: before that group or request
    int32_t own, at;
    int32_t team, lane, width;
};

// What a tile of a prefix, an own key of a kv head, and a request and kv head take a CTA of the bf16 kernels (an SM's
// share for the latter two): 512 bytes a key at some 75 GB/s an SM.
constexpr float kPrefixTileUs = 1.6f, kOwnKeyUs = 512.f / 75e3f, kOwnItemUs = 2.f;

// Every CTA of the first launch works out the whole plan (a few loads a group and request); CTA 0 writes it
// down.  `run` and `sums` (kThreads / 32) are in shared memory.
template <int kThreads>
__device__ void prefix_make_plan(const PrefixAttentionArgs &a, const PrefixCut &cut, PrefixRun &run, int64_t *sums) {
    const int32_t Ng = a.num_groups, B = a.cache.batch, Hkv = a.num_kv_heads, tid = threadIdx.x;
    const int32_t each = (Ng + kThreads - 1) / kThreads, g0 = min(tid * each, Ng), g1 = min(g0 + each, Ng);
    const int32_t own_each = (B + kThreads - 1) / kThreads, b0 = min(tid * own_each, B), b1 = min(b0 + own_each, B);
    const PrefixSpace s = prefix_space(a);
    int64_t before = 0, own_before = 0, all = 0, own_all = 0, own_keys = 0;
    bool falls = false, mine = false;
    // the first time the work of this thread's groups and requests is summed up, the second time each gets its place
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const bool write = pass == 1 && blockIdx.x == 0;
        int64_t units = 0, own_units = 0;
        if (pass == 0 || write || (mine && !run.own))
            for (int32_t g = g0; g < g1; ++g) {
                const PrefixGroup x = prefix_group(a, cut, g);
                const int64_t n = (int64_t)Hkv * ((x.items + cut.width - 1) / cut.width) * (x.tiles + kPrefixExtra);
                falls |= x.r1 < x.r0;
                if (x.ok) own_keys -= (int64_t)x.len * (x.r1 - x.r0);
                if (pass == 1 && mine && !run.own && run.from >= before + units && run.from < before + units + n) {
                    run.at = g;
                    run.units = before + units;
                }
                if (write) s.units[g] = before + units;
                units += n;
            }
        if (cut.own_apart) {  // how many own keys there are, for the CTAs that they get
            if (pass == 0)
                for (int32_t b = b0; b < b1; ++b) {
                    const int32_t row = a.cache.slot[b];
                    if ((uint32_t)row < (uint32_t)a.cache.table_rows) own_keys += a.cache.kv_len[row];
                }
        } else if (b0 < b1 && (pass == 0 || write || (mine && run.own))) {
            int32_t g = prefix_group_of(a, b0);
            PrefixGroup x = prefix_group(a, cut, g);
            for (int32_t b = b0; b < b1; ++b) {
                while (b >= x.r1 && g + 1 < Ng) x = prefix_group(a, cut, ++g);
                const PrefixRequest r = prefix_request(a, cut, x, b);
                const int64_t n = (int64_t)Hkv * r.items * (r.tiles + kOwnExtra);
                if (pass == 1 && mine && run.own && run.from >= own_before + own_units && run.from < own_before + own_units + n) {
                    run.at = b;
                    run.units = own_before + own_units;
                }
                if (write) s.own_units[b] = own_before + own_units;
                own_units += n;
            }
        }
        if (pass == 1) break;
        before = prefix_scan<kThreads>(units, sums, &all);
        if (cut.own_apart) prefix_scan<kThreads>(own_keys, sums, &own_keys);
        else own_before = prefix_scan<kThreads>(own_units, sums, &own_all);
        falls = __syncthreads_or(falls);
        if (falls) all = own_all = 0;
        if (tid == 0) {
            // The CTAs of either kind; every one has a unit, so that the parts of an item lie in neighbouring runs.  Own
            // keys in a launch of their own: the time that their CTAs need, next to that of the prefixes (1.6 us a tile).
            const float work = (float)all * (float)cut.width * (cut.own_apart ? kPrefixTileUs : 1.f);
            const float own_work = cut.own_apart ? kOwnKeyUs * (float)max(own_keys, (int64_t)0) * (float)Hkv + kOwnItemUs * (float)B * (float)Hkv
                                                 : (float)own_all;
            int32_t teams = 0;
            if (all > 0) {
                teams = max(1, (int32_t)((float)cut.ctas * work / (work + own_work) / (float)cut.width + 0.5f));
                teams = min(teams, (cut.ctas - (own_all > 0)) / cut.width);
                teams = (int32_t)min((int64_t)teams, all);
            }
            const int32_t own_ctas = (int32_t)min((int64_t)(cut.ctas - teams * cut.width), own_all);
            run.width = cut.width;
            run.own = (int32_t)blockIdx.x >= teams * cut.width;
            run.team = run.own ? (int32_t)blockIdx.x - teams * cut.width : (int32_t)blockIdx.x / cut.width;
            run.lane = run.own ? 0 : (int32_t)blockIdx.x % cut.width;
            run.from = run.to = 0;
            if (!run.own) {
                run.from = prefix_cut_at(all, run.team, teams);
                run.to = prefix_cut_at(all, run.team + 1, teams);
            } else if (run.team < own_ctas) {
                run.from = prefix_cut_at(own_all, run.team, own_ctas);
                run.to = prefix_cut_at(own_all, run.team + 1, own_ctas);
            }
            if (blockIdx.x == 0)
                *static_cast<PrefixPlan *>(a.workspace) = PrefixPlan{all, own_all, falls, cut.width, teams, own_ctas};
        }
        __syncthreads();
        mine = run.from < run.to;
    }
    __syncthreads();
}

// One stretch of a CTA's run: key tiles [tile, tile + count) of one item.
struct PrefixStretch {
    int32_t own;                 // its kind
    int32_t first, tokens;       // of the group or request
    int32_t row;                 // of the table
    int32_t from, len;           // keys [from, len)
    int32_t h, index, items;     // kv head; number of the row tile and how many there are (none past the last)
    int32_t tile, count;         // tile 0: that of key `from`
    bool goes_on;                // with an item that another CTA started: the part goes to the CTA's slot
};

// Walks the stretches of a run.  A whole warp calls it, all lanes together; every warp gets the same answers.  Items
// of one group or request and kv head after kv head come by counting; a division is taken where it begins.
struct PrefixWalk {
    int64_t u, units;
    int32_t at;                     // the group or request at hand, from unit `units` on
    int32_t inside = 0, item = -1;  // unit of its item `item`; -1: not begun
    int32_t per, items;             // units of an item, items of all kv heads
    PrefixStretch now;              // what its items share
    int32_t h, index;
    // lane l: request base + l and the units of all up to it
    int32_t base = -1;
    PrefixRequest mine;
    int64_t sum = 0;

    __device__ __forceinline__ explicit PrefixWalk(const PrefixRun &run) : u(run.from), units(run.units), at(run.at) {}
    __device__ __forceinline__ bool next(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run,
                                         PrefixStretch &s) {
        while (u < run.to) {
            if (item < 0 && !(run.own ? begin_request(a, cut) : begin_group(a, cut, run))) {
                u = run.to;  // (never: u < run.to <= all units)
                return false;
            }
            const int32_t extra = run.own ? kOwnExtra : kPrefixExtra;
            const int32_t end = (int32_t)min((int64_t)per, inside + (run.to - u));
            s = now;
            s.goes_on = inside > extra;
            s.tile = max(0, inside - extra);
            s.count = end - extra - s.tile;
            s.h = h;
            s.index = run.own ? index : index * run.width + run.lane;
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
    int32_t wide;  // items of a kv head
    // The place of unit u in what begins at `units`.
    __device__ __forceinline__ void place(const PrefixAttentionArgs &a, int32_t extra, int32_t tiles) {
        per = tiles + extra;
        items = a.num_kv_heads * wide;
        const int64_t x = u - units;
        item = (int32_t)prefix_div(x, per);
        inside = (int32_t)(x - (int64_t)item * per);
        h = item / wide;
        index = item - h * wide;
    }
    __device__ __forceinline__ bool begin_group(const PrefixAttentionArgs &a, const PrefixCut &cut, const PrefixRun &run) {
        for (; at < a.num_groups; ++at) {
            const PrefixGroup x = prefix_group(a, cut, at);
            wide = (x.items + run.width - 1) / run.width;
            const int64_t n = (int64_t)a.num_kv_heads * wide * (x.tiles + kPrefixExtra);
            if (u < units + n) {
                now.own = 0;
                now.first = x.first; now.tokens = x.tokens; now.row = x.row; now.from = 0; now.len = x.len;
                now.items = x.items;
                place(a, kPrefixExtra, x.tiles);
                return true;
            }
            units += n;
        }
        return false;
    }
    __device__ __forceinline__ bool begin_request(const PrefixAttentionArgs &a, const PrefixCut &cut) {
        constexpr uint32_t kAll = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        while (true) {
            if (base < 0 || at >= base + 32) {
                if (at >= a.cache.batch) return false;
                base = at;
                mine = PrefixRequest{};
                if (base + lane < a.cache.batch)
                    mine = prefix_request(a, cut, prefix_group(a, cut, prefix_group_of(a, base + lane)), base + lane);
                sum = (int64_t)a.num_kv_heads * mine.items * (mine.tiles + kOwnExtra);
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int64_t y = __shfl_up_sync(kAll, sum, off);
                    if (lane >= off) sum += y;
                }
                sum += units;  // units up to the end of this lane's request
            }
            const uint32_t holds = __ballot_sync(kAll, u < sum);
            if (holds == 0) {
                units = __shfl_sync(kAll, sum, 31);
                at = base + 32;
                continue;
            }
            const int src = __ffs(holds) - 1;
            at = base + src;
            const int32_t tiles = __shfl_sync(kAll, mine.tiles, src);
            wide = __shfl_sync(kAll, mine.items, src);
            units = __shfl_sync(kAll, sum, src) - (int64_t)a.num_kv_heads * wide * (tiles + kOwnExtra);
            now.own = 1;
            now.first = __shfl_sync(kAll, mine.first, src);
            now.tokens = __shfl_sync(kAll, mine.n, src);
            now.row = __shfl_sync(kAll, mine.row, src);
            now.from = __shfl_sync(kAll, mine.from, src);
            now.len = __shfl_sync(kAll, mine.len, src);
            now.items = wide;
            place(a, kOwnExtra, tiles);
            return true;
        }
    }
};

// A row's place in the CTAs' slots: item and row of its tile.
struct PrefixPlace {
    int32_t index, row;
};
__device__ __forceinline__ PrefixPlace prefix_place(const PrefixCut &cut, int32_t token, int32_t head, int32_t tile) {
    if (cut.by_rows) {
        const int32_t row = token * cut.G + head;  // (T * Hq < 2^31)
        return PrefixPlace{row / tile, row % tile};
    }
    const int32_t index = token / tile, t = token - index * tile, half = t / cut.own_tile;  // row tiles of own_tile tokens
    return PrefixPlace{index, half * 128 + (t - half * cut.own_tile) * cut.G + head};
}
// The CTAs that have parts of an item which starts at unit u: the first, and how many go on with it.
struct PrefixParts {
    int32_t cta, more, step;
};
__device__ __forceinline__ PrefixParts prefix_parts(const PrefixPlan &plan, int64_t u, int32_t tiles, int32_t lane) {
    const int32_t t0 = prefix_team(plan.units, u + kPrefixExtra, plan.teams);
    return PrefixParts{t0 * plan.width + lane, prefix_team(plan.units, u + kPrefixExtra + tiles - 1, plan.teams) - t0, plan.width};
}
__device__ __forceinline__ PrefixParts own_parts(const PrefixPlan &plan, int64_t u, int32_t tiles) {
    const int32_t t0 = prefix_team(plan.own_units, u + kOwnExtra, plan.own_ctas);
    return PrefixParts{plan.teams * plan.width + t0, prefix_team(plan.own_units, u + kOwnExtra + tiles - 1, plan.own_ctas) - t0, 1};
}

PrefixCut prefix_cut_rows(const PrefixAttentionArgs &a);
PrefixCut prefix_cut_tc(const PrefixAttentionArgs &a);
cudaError_t launch_prefix_rows(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);
cudaError_t launch_prefix_tc(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);
cudaError_t launch_prefix_own(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream);

}  // namespace kda
