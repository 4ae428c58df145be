// Attention over a shared prefix: the work in fp32 on the FMA units (for fp32, and for bf16 with a scale of 0
// or below), the join of the parts, and the choice between the FMA and the tensor-core kernels.
// kda_attention_rows.cuh computes a tile of 32 rows and 64 keys.
#include <cfloat>

#include "kda_attention_rows.cuh"
#include "kda_prefix_attention.cuh"

namespace kda {
namespace {

using rows::kRows;
using rows::kSmem;
using rows::kThreads;
using rows::kTile;

// Prefixes: two CTAs an SM, items of 32 rows of a group.  Bound by a tile's chain, some 8 us (pages, loads, 4,096 FMAs a
// thread): three prompts of up to 777 tokens x 5 branches 13 us.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) prefix_rows_kernel(const PrefixAttentionArgs a, const PrefixCut cut) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    __shared__ PrefixRun run;
    __shared__ int64_t sums[2 * kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t G = cut.G;
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);
    const PrefixSpace space = prefix_space(a);
    grid_wait();
    prefix_begin(a, space);
    prefix_make_plan<kThreads>(a, cut, run, sums);
    PrefixWalk walk(run);
    PrefixStretch s;
    while (walk.next(a, cut, run, s)) {
        const int32_t r0 = s.index * kRows, num_rows = s.tokens * G;
        const auto place = [&](int r) {  // row r of the tile, as a row of [T][Hq]
            return (int64_t)(s.first + (r0 + r) / G) * a.num_q_heads + s.h * G + (r0 + r) % G;
        };
        __syncthreads();  // the last stretch's products have read q
        rows::load_q(tiles_of, [&](int r) -> const T * { return r0 + r < num_rows ? q + place(r) * kD : nullptr; });
        rows::State st;
        for (int32_t i = 0; i < s.count; ++i)
            rows::tile(tiles_of, s_keys, st, pool, a.cache, a.num_kv_heads, s.h, s.row, (s.tile + i) * kTile, s.len, a.scale,
                       [&](int, int32_t j) { return j < s.len; });
        float *slot = prefix_slot(space, cut, (int32_t)blockIdx.x), *to = s.goes_on ? slot : space.o;
        float2 *ml = s.goes_on ? prefix_slot_ml(slot, cut) : space.ml;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r0 + r >= num_rows) continue;
            const int64_t at = s.goes_on ? r : place(r);
            store4(to + at * kD + 4 * tx, make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]));
            store4(to + at * kD + 64 + 4 * tx, make_float4(st.o[i][4], st.o[i][5], st.o[i][6], st.o[i][7]));
            if (tx != 0) continue;
            ml[at] = make_float2(st.m[i], st.l[i]);
            // (a token whose query heads lie in two items gets what either says for its own heads: by query head)
            if (!s.goes_on) space.more[at] = make_int4((int32_t)blockIdx.x, s.more, 1, r);
        }
    }
    if (threadIdx.x == 0) space.done[blockIdx.x] = !run.bad;
}

// Own keys: a CTA a request, kv head and 32 rows (and further ones where a request has more than most).  Tiles begin
// with the first own key, not on a boundary: up to 60 own keys are then one tile instead of two (20 us a call, not 28).
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) prefix_own_rows_kernel(const PrefixAttentionArgs a, const PrefixCut cut) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t G = cut.G, b = blockIdx.x, h = blockIdx.y;
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join comes up when the last CTA has
    const PrefixRequest req = prefix_request(a, cut, b);
    if (!req.ok && blockIdx.z == 0 && h == 0 && threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)b);
    const PrefixSpace space = prefix_space(a);
    const int32_t num_rows = req.n * G, p0 = req.len - req.n;
    for (int32_t r0 = blockIdx.z * kRows; r0 < num_rows; r0 += gridDim.z * kRows) {
        const auto place = [&](int r) {
            return (int64_t)(req.first + (r0 + r) / G) * a.num_q_heads + h * G + (r0 + r) % G;
        };
        __syncthreads();  // the last rows' products have read q
        rows::load_q(tiles_of, [&](int r) -> const T * { return r0 + r < num_rows ? q + place(r) * kD : nullptr; });
        int32_t p[4];  // indices of this thread's rows (past the last row: -1 sees nothing)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = r0 + 4 * ty + i < num_rows ? p0 + (r0 + 4 * ty + i) / G : -1;
        rows::State st;
        const int32_t end = p0 + (min(r0 + kRows, num_rows) - 1) / G + 1;  // no row sees a key from here on
        const int32_t tiles = (int32_t)(((uint32_t)(end - req.from) + kTile - 1) / kTile);
        for (int32_t t = 0; t < tiles; ++t)
            rows::tile(tiles_of, s_keys, st, pool, a.cache, a.num_kv_heads, h, req.row, req.from + t * kTile, end, a.scale,
                       [&](int i, int32_t j) { return j <= p[i]; });
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r0 + r >= num_rows) continue;
            const int64_t at = place(r);
            store4(space.own_o + at * kD + 4 * tx, make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]));
            store4(space.own_o + at * kD + 64 + 4 * tx, make_float4(st.o[i][4], st.o[i][5], st.o[i][6], st.o[i][7]));
            if (tx == 0) space.own[at] = make_float4(st.m[i], st.l[i], req.from > 0, 0.f);
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) grid_wait();  // the launch ends after the one before it
}

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

// What some parts come to, four channels a lane.  A maximum m stands for 2^(c m).
struct Joined {
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 ml, float4 y, float c) {
        const float now = fmaxf(top, ml.x);
        const auto weight = [&](float m, float l) {  // of a part without keys 0, but a NaN sum stays one
            return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : tc::ex2_approx((m - now) * c);
        };
        const float keep = weight(top, sum), w = weight(ml.x, ml.y);
        top = now;
        sum = fmaf(sum, keep, w * ml.y);
        o = make_float4(fmaf(o.x, keep, w * y.x), fmaf(o.y, keep, w * y.y), fmaf(o.z, keep, w * y.z), fmaf(o.w, keep, w * y.w));
    }
};

// kWarps warps a row of [T][Hq], which take its parts in turns.  Bound by rounds of loads one after the other (where the
// row's parts lie; the parts, four at a time): 24,576 rows of two or three parts 15 us, most of it from L2.  With each
// row's parts worked out from the plan again instead of looked up: 22 us.
template <typename T, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixAttentionArgs a, const PrefixCut cut, float c) {
    constexpr int kRowsCta = kJoinThreads / 32 / kWarps;
    __shared__ float4 s_o[kJoinThreads / 32][32];
    __shared__ float2 s_ml[kJoinThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = warp % kWarps;
    const int64_t row = (int64_t)blockIdx.x * kRowsCta + warp / kWarps;
    const PrefixSpace space = prefix_space(a);
    const bool live = row < (int64_t)a.cache.total_tokens * a.num_q_heads;
    const int32_t token = live ? (int32_t)(row / a.num_q_heads) : 0, head = live ? (int32_t)(row - (int64_t)token * a.num_q_heads) : 0;
    const int64_t more_at = cut.by_rows ? row : (int64_t)token * a.num_kv_heads + head / cut.G;
    grid_wait();
    // (all that may be wanted at once; what nothing was written to is not used)
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool first = live && turn == 0;
    const float4 own = live ? space.own[row] : make_float4(0.f, -1.f, 0.f, 0.f);
    const int4 more = live ? space.more[more_at] : make_int4(0, 0, 0, 0);
    const float4 own_o = first ? load4(space.own_o + row * kD + 4 * lane) : none, o = first ? load4(space.o + row * kD + 4 * lane) : none;
    const float2 ml = first ? space.ml[row] : make_float2(-INFINITY, 0.f);
    // Where a CTA of the first launch gave up (and said so), nothing is joined: where parts lie may be unsaid.
    bool lost = false;
    for (int32_t i = threadIdx.x; i < cut.ctas; i += kJoinThreads) lost |= space.done[i] != 1;
    if (__syncthreads_or(lost)) return;
    const bool wanted = !(own.y < 0.f);  // (else the row has no result; a NaN sum is one)
    Joined x;
    if (wanted && turn == 0) {
        x.top = own.x;
        x.sum = own.y;
        x.o = own_o;
    }
    if (wanted && own.z != 0.f) {
        const int32_t r = more.w + (cut.by_rows ? 0 : head % cut.G);
        if (turn == 0) x.add(ml, o, c);
        for (int32_t k0 = 1 + turn; k0 <= more.y; k0 += 4 * kWarps) {  // four parts' loads at a time
            float2 mls[4];
            float4 ys[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mls[k] = make_float2(-INFINITY, 0.f);
                ys[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k * kWarps > more.y) continue;
                float *slot = prefix_slot(space, cut, more.x + (k0 + k * kWarps) * more.z);
                mls[k] = prefix_slot_ml(slot, cut)[r];
                ys[k] = load4(slot + (int64_t)r * kD + 4 * lane);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) x.add(mls[k], ys[k], c);
        }
    }
    if constexpr (kWarps > 1) {
        s_o[warp][lane] = x.o;
        if (lane == 0) s_ml[warp] = make_float2(x.top, x.sum);
        __syncthreads();
        if (turn != 0) return;
#pragma unroll
        for (int k = 1; k < kWarps; ++k) x.add(s_ml[warp + k], s_o[warp + k][lane], c);
    }
    if (!wanted) return;
    const float inv = x.sum == 0.f ? 0.f : 1.f / x.sum;
    store4(static_cast<T *>(a.o) + row * kD + 4 * lane, make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
}

// Warps a row by how many parts its prefix may come in: an item's key tiles, or the CTAs that an item gets.
// 10 beams behind 32,768 tokens, one kv head (151 parts): 54 us with one, 33 with eight.  64 x 2 tokens behind 131,072
// (up to 5 parts, 8,192 rows): 393 us with one, 405 with four.
template <typename T>
cudaError_t launch_join(const PrefixAttentionArgs &a, const PrefixCut &cut, float c, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.cache.total_tokens * a.num_q_heads, Ng = a.num_groups;
    const int64_t per_group = (a.cache.total_tokens + Ng - 1) / Ng * (cut.by_rows ? cut.G : 1);
    const int64_t items = Ng * a.num_kv_heads * ((per_group + cut.tile - 1) / cut.tile);
    const int64_t tiles = ((int64_t)a.cache.table_width * a.cache.page_size + cut.keys - 1) / cut.keys;
    const int64_t share = cut.ctas / items + 1, parts = share < tiles ? share : tiles;
    const auto launch = [&](auto kernel, int warps) {
        const int64_t per = kJoinThreads / 32 / warps;
        return launch_serial(kernel, dim3((unsigned)((rows + per - 1) / per)), kJoinThreads, 0, stream, a, cut, c);
    };
    if (parts > 16) return launch(prefix_join_kernel<T, 8>, 8);
    return parts > 8 ? launch(prefix_join_kernel<T, 4>, 4) : launch(prefix_join_kernel<T, 1>, 1);
}

template <typename T>
cudaError_t launch_rows(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream) {
    cudaError_t e = allow_smem(prefix_rows_kernel<T>, kSmem);
    if (e == cudaSuccess) e = allow_smem(prefix_own_rows_kernel<T>, kSmem);
    if (e == cudaSuccess) e = launch_serial(prefix_rows_kernel<T>, dim3((unsigned)cut.ctas), kThreads, kSmem, stream, a, cut);
    if (e != cudaSuccess) return e;
    // CTAs for the rows of the longest request, as far as it is not much longer than most
    const int64_t tokens = a.cache.total_tokens, B = a.cache.batch;
    const int64_t most = (a.max_tokens < tokens ? a.max_tokens : tokens) * cut.G, share = 2 * ((tokens + B - 1) / B) * cut.G;
    const int64_t z = ((most < share ? most : share) + kRows - 1) / kRows;
    const dim3 grid((unsigned)B, (unsigned)a.num_kv_heads, (unsigned)(z < 1024 ? z : 1024));
    return launch_serial(prefix_own_rows_kernel<T>, grid, kThreads, kSmem, stream, a, cut);
}

size_t space_bytes(const PrefixAttentionArgs &a, const PrefixCut &cut) {
    PrefixSpace s;
    return prefix_space_at(a, &s) + (size_t)cut.ctas * cut.slot_rows * kSlotRow * sizeof(float);
}

}  // namespace

PrefixCut prefix_cut_rows(const PrefixAttentionArgs &a, int32_t sms) {
    return PrefixCut{1, a.num_q_heads / a.num_kv_heads, kRows, kTile, 2 * sms, kRows, 1, 8.f};
}

// (bf16: of either kind of kernels, as the scale decides; whatever GPU the call runs on)
size_t prefix_attention_workspace(kda_dtype dtype, int32_t batch, int32_t total_tokens, int32_t num_groups,
                                  int32_t num_q_heads, int32_t num_kv_heads) {
    PrefixAttentionArgs a{};
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.num_groups = num_groups;
    a.cache.batch = batch;
    a.cache.total_tokens = total_tokens;
    const size_t rows = space_bytes(a, prefix_cut_rows(a, kPrefixSms)), tc = space_bytes(a, prefix_cut_tc(a, kPrefixSms));
    return dtype == KDA_BF16 && tc > rows ? tc : rows;
}

cudaError_t launch_prefix_attention(const PrefixAttentionArgs &a, cudaStream_t stream) {
    if (a.cache.total_tokens == 0) return cudaSuccess;
    // The tensor-core kernels keep their running maximum on unscaled scores, in the order that a positive scale
    // leaves alone; any other scale (and fp32) runs on the FMA units.
    constexpr double kLog2e = 1.4426950408889634;
    const int32_t sms = device_sm_count() < kPrefixSms ? device_sm_count() : kPrefixSms;
    if (a.dtype == KDA_BF16 && a.scale > 0.f && a.scale <= FLT_MAX) {
        const PrefixCut cut = prefix_cut_tc(a, sms);
        cudaError_t e = launch_prefix_tc(a, cut, stream);
        if (e == cudaSuccess) e = launch_prefix_own(a, cut, stream);
        return e == cudaSuccess ? launch_join<__nv_bfloat16>(a, cut, (float)((double)a.scale * kLog2e), stream) : e;
    }
    const PrefixCut cut = prefix_cut_rows(a, sms);
    if (a.dtype == KDA_BF16) {
        const cudaError_t e = launch_rows<__nv_bfloat16>(a, cut, stream);
        return e == cudaSuccess ? launch_join<__nv_bfloat16>(a, cut, (float)kLog2e, stream) : e;
    }
    const cudaError_t e = launch_rows<float>(a, cut, stream);
    return e == cudaSuccess ? launch_join<float>(a, cut, (float)kLog2e, stream) : e;
}

}  // namespace kda
