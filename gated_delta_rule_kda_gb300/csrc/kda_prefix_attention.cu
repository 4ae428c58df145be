// Attention over a shared prefix: the work in fp32 on the FMA units (for fp32, and for bf16 with a scale of 0
// or below), the join of the parts, and the choice between the FMA and the tensor-core kernel.
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

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) prefix_rows_kernel(const PrefixAttentionArgs a, const PrefixCut cut) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    __shared__ PrefixRun run;
    __shared__ int64_t sums[kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t G = cut.G;
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);
    grid_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    prefix_make_plan<kThreads>(a, cut, run, sums);
    const PrefixSpace space = prefix_space(a);
    PrefixWalk walk(run);
    PrefixStretch s;
    while (walk.next(a, cut, run, s)) {
        const int32_t r0 = s.index * kRows, num_rows = s.tokens * G;
        const auto place = [&](int r) {  // row r of the tile, as a row of [T][Hq]
            return (int64_t)(s.first + (r0 + r) / G) * a.num_q_heads + s.h * G + (r0 + r) % G;
        };
        __syncthreads();  // the last stretch's products have read q
        rows::load_q(tiles_of, [&](int r) -> const T * { return r0 + r < num_rows ? q + place(r) * kD : nullptr; });
        int32_t p[4];  // the last key that this thread's rows see (past the last row: none)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t row = r0 + 4 * ty + i;
            p[i] = row >= num_rows ? -1 : s.own ? s.len - s.tokens + row / G : s.len - 1;
        }
        rows::State st;
        for (int32_t i = 0; i < s.count; ++i)
            rows::tile(tiles_of, s_keys, st, pool, a.cache, a.num_kv_heads, s.h, s.row,
                       (s.from / kTile + s.tile + i) * kTile, s.len, a.scale,
                       [&](int k, int32_t j) { return j >= s.from && j <= p[k]; });
        const PrefixPart to = s.goes_on ? prefix_slot(space, cut, (int32_t)blockIdx.x) : prefix_part(space, s.own);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r0 + r >= num_rows) continue;
            const int64_t at = s.goes_on ? r : place(r);
            *reinterpret_cast<float4 *>(to.o + at * kD + 4 * tx) = make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]);
            *reinterpret_cast<float4 *>(to.o + at * kD + 64 + 4 * tx) = make_float4(st.o[i][4], st.o[i][5], st.o[i][6], st.o[i][7]);
            if (tx == 0) to.ml[at] = make_float2(st.m[i], st.l[i]);
        }
    }
    if (threadIdx.x == 0) space.done[blockIdx.x] = 1;
}

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;

// Rows (token, query head) of request blockIdx.x and kv head blockIdx.y, a warp each in turn, four channels a lane.
// c: 2^(c m) is what a maximum m of the parts stands for.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixAttentionArgs a, const PrefixCut cut, float c) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t b = blockIdx.x, h = blockIdx.y, G = cut.G, first_row = blockIdx.z * (kJoinThreads / 32) + warp;
    // (the request's sizes are inputs of the first launch, which began after all before it was done)
    const int32_t g = prefix_group_of(a, b);
    const PrefixGroup x = prefix_group(a, cut, g);
    const PrefixRequest r = prefix_request(a, cut, x, b);
    if (!r.ok && h == 0 && blockIdx.z == 0 && threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)b);
    const PrefixSpace space = prefix_space(a);
    const PrefixPart own = prefix_part(space, 1), shared = prefix_part(space, 0);
    grid_wait();
    const PrefixPlan plan = *static_cast<const PrefixPlan *>(a.workspace);
    if (plan.bad) {
        if (r.ok && h == 0 && blockIdx.z == 0 && threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)b);
        return;
    }
    const int64_t units = x.items > 0 ? space.units[g] : 0, own_units = r.items > 0 && !cut.own_apart ? space.own_units[b] : 0;
    for (int32_t row = first_row; row < r.n * G; row += gridDim.z * (kJoinThreads / 32)) {
        const int32_t token = row / G, head = row - token * G;
        const int64_t q_row = (int64_t)(r.first + token) * a.num_q_heads + h * G + head;
        // its parts: own keys, what goes on with them, the prefix, what goes on with that
        const PrefixPlace mine = prefix_place(cut, token, head, cut.own_tile);
        PrefixParts own_in{-1, 0, 0};  // (a launch of its own leaves one part)
        if (!cut.own_apart)
            own_in = own_parts(plan, own_units + ((int64_t)h * r.items + mine.index) * (r.tiles + kOwnExtra), r.tiles);
        PrefixPlace at{0, 0};
        PrefixParts in{0, -1, 0};
        if (x.items > 0) {
            at = prefix_place(cut, r.first - x.first + token, head, cut.tile);
            const int32_t wide = (x.items + plan.width - 1) / plan.width, item = h * wide + at.index / plan.width;
            in = prefix_parts(plan, units + (int64_t)item * (x.tiles + kPrefixExtra), x.tiles, at.index % plan.width);
        }
        const int32_t parts = 2 + own_in.more + in.more;
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        bool lost = false;
        for (int32_t k0 = 0; k0 < parts; k0 += 32) {
            const int32_t k = k0 + lane;
            float2 ml = make_float2(-INFINITY, 0.f);
            const float *o = own.o;
            if (k < parts) {
                const int32_t j = k - own_in.more - 1;  // of the prefix's parts, from 0 on
                const int32_t cta = j < 0 ? own_in.cta + k : in.cta + j * in.step;
                lost |= cta >= 0 && space.done[cta] != 1;
                const bool dense = k == 0 || j == 0;
                const PrefixPart part = dense ? (j < 0 ? own : shared) : prefix_slot(space, cut, cta);
                const int64_t place = dense ? q_row : j < 0 ? mine.row : at.row;
                ml = part.ml[place];
                o = part.o + place * kD;
            }
            lost |= ml.y < 0.f;  // (marked)
            if (__any_sync(kAll, lost)) break;  // a launch before this one gave up (and said so)
            float now = ml.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) now = fmaxf(now, __shfl_xor_sync(kAll, now, off));
            now = fmaxf(now, top);
            const auto weight = [&](float m, float l) {  // (a NaN sum stays one)
                return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : tc::ex2_approx((m - now) * c);
            };
            const float keep = weight(top, sum), w = weight(ml.x, ml.y);
            top = now;
            float s = w * ml.y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kAll, s, off);
            sum = fmaf(sum, keep, s);
            acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
            const int32_t here = min(parts - k0, 32);
#pragma unroll 4
            for (int32_t i = 0; i < here; ++i) {
                const float wi = __shfl_sync(kAll, w, i);
                const float *oi = reinterpret_cast<const float *>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(o), i));
                const float4 y = *reinterpret_cast<const float4 *>(oi + 4 * lane);
                acc = make_float4(fmaf(wi, y.x, acc.x), fmaf(wi, y.y, acc.y), fmaf(wi, y.z, acc.z), fmaf(wi, y.w, acc.w));
            }
        }
        if (__any_sync(kAll, lost)) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4(static_cast<T *>(a.o) + q_row * kD + 4 * lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
}

template <typename T>
cudaError_t launch_join(const PrefixAttentionArgs &a, const PrefixCut &cut, float c, cudaStream_t stream) {
    // CTAs for the rows of the longest request, as far as it is not much longer than most: 16 rows each
    const int64_t T_ = a.cache.total_tokens, B = a.cache.batch;
    const int64_t most = (a.max_tokens < T_ ? a.max_tokens : T_) * cut.G, share = 2 * ((T_ + B - 1) / B) * cut.G;
    const int64_t z = ((most < share ? most : share) + 15) / 16;
    const dim3 grid((unsigned)B, (unsigned)a.num_kv_heads, (unsigned)(z < 256 ? z : 256));
    return launch_serial(prefix_join_kernel<T>, grid, kJoinThreads, 0, stream, a, cut, c);
}

size_t space_bytes(const PrefixAttentionArgs &a, const PrefixCut &cut) {
    const size_t parts = 2 * (size_t)prefix_part_floats((int64_t)a.cache.total_tokens * a.num_q_heads);
    return prefix_parts_at(a.num_groups, a.cache.batch) +
           (parts + (size_t)cut.ctas * cut.slot_rows * (kD + 2)) * sizeof(float);
}

}  // namespace

PrefixCut prefix_cut_rows(const PrefixAttentionArgs &a) {
    return PrefixCut{1, a.num_q_heads / a.num_kv_heads, kRows, kRows, kTile, kPrefixCtas, kRows, 1, 0};
}

cudaError_t launch_prefix_rows(const PrefixAttentionArgs &a, const PrefixCut &cut, cudaStream_t stream) {
    const auto kernel = a.dtype == KDA_BF16 ? prefix_rows_kernel<__nv_bfloat16> : prefix_rows_kernel<float>;
    const cudaError_t e = allow_smem(kernel, kSmem);
    return e == cudaSuccess ? launch_serial(kernel, dim3((unsigned)cut.ctas), kThreads, kSmem, stream, a, cut) : e;
}

// (bf16: of either kernel, as the scale decides)
size_t prefix_attention_workspace(kda_dtype dtype, int32_t batch, int32_t total_tokens, int32_t num_groups,
                                  int32_t num_q_heads, int32_t num_kv_heads) {
    PrefixAttentionArgs a{};
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.num_groups = num_groups;
    a.cache.batch = batch;
    a.cache.total_tokens = total_tokens;
    const size_t rows = space_bytes(a, prefix_cut_rows(a)), tc = space_bytes(a, prefix_cut_tc(a));
    return dtype == KDA_BF16 && tc > rows ? tc : rows;
}

cudaError_t launch_prefix_attention(const PrefixAttentionArgs &a, cudaStream_t stream) {
    if (a.cache.total_tokens == 0) return cudaSuccess;
    // The tensor-core kernel keeps its running maximum on unscaled scores, in the order that a positive scale
    // leaves alone; any other scale (and fp32) runs on the FMA units.
    const bool tensor = a.dtype == KDA_BF16 && a.scale > 0.f && a.scale <= FLT_MAX;
    const PrefixCut cut = tensor ? prefix_cut_tc(a) : prefix_cut_rows(a);
    cudaError_t e = tensor ? launch_prefix_tc(a, cut, stream) : launch_prefix_rows(a, cut, stream);
    if (e == cudaSuccess && tensor) e = launch_prefix_own(a, cut, stream);
    if (e != cudaSuccess) return e;
    constexpr double kLog2e = 1.4426950408889634;
    const float c = tensor ? (float)((double)a.scale * kLog2e) : (float)kLog2e;
    return a.dtype == KDA_BF16 ? launch_join<__nv_bfloat16>(a, cut, c, stream) : launch_join<float>(a, cut, c, stream);
}

}  // namespace kda
