// Attention over a shared prefix in fp32 on the FMA units: the two launches of kda_prefix_attention for
// fp32, and for bf16 with a scale of 0 or below.
//
//   prefix:  partial (o, m, l) of 32 rows of a group over a stretch of its prefix's key tiles
//   own:     (o, m, l) of 32 rows of a request over its own keys, then joined with its prefix's parts:
//            M = max m_i;  o = (sum_i e^(m_i - M) o_i) / (sum_i e^(m_i - M) l_i)
// kda_attention_rows.cuh computes a tile.
#include <cfloat>

#include "kda_attention_rows.cuh"
#include "kda_prefix_attention.cuh"

namespace kda {
namespace {

using rows::kRows;
using rows::kSmem;
using rows::kThreads;
using rows::kTile;

constexpr int kCtas = kPrefixCtas;  // two an SM

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) prefix_rows_kernel(const PrefixAttentionArgs a, const PrefixCut cut) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    __shared__ PrefixRun run;
    __shared__ int64_t sums[kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t G = a.num_q_heads / a.num_kv_heads;
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);
    grid_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    prefix_make_plan<kThreads>(a, cut, run, sums);
    PrefixWalk walk(a, cut, run);
    PrefixStretch s;
    while (walk.next(a, cut, run, s)) {
        if (s.index >= s.items) continue;
        __syncthreads();  // the last stretch's products have read q
        rows::load_q(tiles_of, [&](int r) -> const T * {
            const int32_t row = s.index * kRows + r, token = row / G;
            return token < s.tokens ? q + ((int64_t)(s.first + token) * a.num_q_heads + s.h * G + row % G) * kD : nullptr;
        });
        rows::State st;
        for (int32_t i = s.tile; i < s.tile + s.count; ++i)
            rows::tile(tiles_of, s_keys, st, pool, a.cache, a.num_kv_heads, s.h, s.row, i * kTile, s.len, a.scale,
                       [&](int, int32_t j) { return j < s.len; });
        float *slot = prefix_slot(a, kRows, s.slot);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * ty + i;
            *reinterpret_cast<float4 *>(slot + kD * row + 4 * tx) = make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]);
            *reinterpret_cast<float4 *>(slot + kD * row + 64 + 4 * tx) = make_float4(st.o[i][4], st.o[i][5], st.o[i][6], st.o[i][7]);
            if (tx == 0) *reinterpret_cast<float2 *>(slot + kD * kRows + 2 * row) = make_float2(st.m[i], st.l[i]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) prefix_own_rows_kernel(const PrefixAttentionArgs a, const PrefixCut cut) {
    extern __shared__ float4 smem4[];
    const rows::Tiles tiles_of(smem4);
    __shared__ rows::Keys s_keys;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t G = a.num_q_heads / a.num_kv_heads, h = blockIdx.y;
    const T *q = static_cast<const T *>(a.q), *pool = static_cast<const T *>(a.kv_pool);
    bool bad;
    const PrefixRequest r = prefix_request(a, cut, (int32_t)blockIdx.x, &bad);
    if (bad && blockIdx.z == 0 && h == 0 && threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, blockIdx.x);
    const AttnRequest &req = r.req;
    const int32_t num_rows = req.n * G, p0 = req.len - req.n;
    for (int32_t r0 = blockIdx.z * kRows; r0 < num_rows; r0 += gridDim.z * kRows) {
        __syncthreads();  // the last rows' products have read q
        rows::load_q(tiles_of, [&](int i) -> const T * {
            const int32_t row = r0 + i;
            return row < num_rows ? q + ((int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G) * kD : nullptr;
        });
        int32_t p[4];  // indices of this thread's rows (past the last row: -1 sees nothing)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = r0 + 4 * ty + i < num_rows ? p0 + (r0 + 4 * ty + i) / G : -1;
        rows::State st;
        const int32_t end = p0 + (min(r0 + kRows, num_rows) - 1) / G + 1;  // no row sees a key from here on
        for (int32_t j0 = r.x.len / kTile * kTile; j0 < end; j0 += kTile) {
            rows::tile(tiles_of, s_keys, st, pool, a.cache, a.num_kv_heads, h, req.row, j0, end, a.scale,
                       [&](int i, int32_t j) { return j >= r.x.len && j <= p[i]; });
            if (j0 > 0x7fffffff - kTile) break;
        }
        grid_wait();  // the prefix's parts are there
        const PrefixPlan plan = *prefix_plan(a);
        if (plan.units < 0) {  // groups that overlap: nothing was computed
            if (threadIdx.x == 0 && h == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, blockIdx.x);
            return;
        }
        const PrefixBase base = prefix_bases(a)[r.g];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t row = r0 + 4 * ty + i;
            if (row >= num_rows) continue;
            const int32_t in_group = (req.first - r.x.first) * G + row;  // (T * Hq < 2^31)
            const PrefixSlots slots = prefix_slots(plan, base, r.x, h, in_group / kRows);
            float m = st.m[i], l = st.l[i];
            float4 x = make_float4(st.o[i][0], st.o[i][1], st.o[i][2], st.o[i][3]);
            float4 y = make_float4(st.o[i][4], st.o[i][5], st.o[i][6], st.o[i][7]);
            for (int32_t k = 0; k < slots.count; ++k) {
                const float *slot = prefix_slot(a, kRows, slots.first + (int64_t)k * slots.step);
                const int at = in_group % kRows;
                const float2 ml = *reinterpret_cast<const float2 *>(slot + kD * kRows + 2 * at);
                const float top = fmaxf(m, ml.x);
                const float w = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : expf(m - top);  // (a NaN sum stays one)
                const float v = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : expf(ml.x - top);
                const float4 px = *reinterpret_cast<const float4 *>(slot + kD * at + 4 * tx);
                const float4 py = *reinterpret_cast<const float4 *>(slot + kD * at + 64 + 4 * tx);
                x = make_float4(w * x.x + v * px.x, w * x.y + v * px.y, w * x.z + v * px.z, w * x.w + v * px.w);
                y = make_float4(w * y.x + v * py.x, w * y.y + v * py.y, w * y.z + v * py.z, w * y.w + v * py.w);
                l = w * l + v * ml.y;
                m = top;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T *dst = static_cast<T *>(a.o) + ((int64_t)(req.first + row / G) * a.num_q_heads + h * G + row % G) * kD;
            store4(dst + 4 * tx, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
            store4(dst + 64 + 4 * tx, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
    }
    grid_wait();  // this grid ends after the one before it, whatever it had to do
}

template <typename T>
cudaError_t launch(const PrefixAttentionArgs &a, cudaStream_t stream) {
    const PrefixCut cut = prefix_cut_rows(a.cache.total_tokens, a.num_groups, a.num_q_heads, a.num_kv_heads);
    cudaError_t e = allow_smem(prefix_rows_kernel<T>, kSmem);
    if (e == cudaSuccess) e = allow_smem(prefix_own_rows_kernel<T>, kSmem);
    if (e == cudaSuccess) e = launch_serial(prefix_rows_kernel<T>, dim3((unsigned)cut.ctas), kThreads, kSmem, stream, a, cut);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.max_tokens * (a.num_q_heads / a.num_kv_heads), tiles = (rows + kRows - 1) / kRows;
    const dim3 grid((unsigned)a.cache.batch, (unsigned)a.num_kv_heads, (unsigned)(tiles < 1024 ? tiles : 1024));
    return launch_serial(prefix_own_rows_kernel<T>, grid, kThreads, kSmem, stream, a, cut);
}

}  // namespace

PrefixCut prefix_cut_rows(int32_t total_tokens, int32_t num_groups, int32_t num_q_heads, int32_t num_kv_heads) {
    const int32_t G = num_q_heads / num_kv_heads;
    const int64_t items = ((int64_t)total_tokens * G / kRows + num_groups) * num_kv_heads;
    return PrefixCut{G, kRows, kTile, kCtas, (int32_t)(items + kCtas < 0x7fffffff ? items + kCtas : 0x7fffffff)};
}

cudaError_t launch_prefix_rows(const PrefixAttentionArgs &a, cudaStream_t stream) {
    return a.dtype == KDA_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

// (bf16: of either pair of launches, as the scale decides)
size_t prefix_attention_workspace(kda_dtype dtype, int32_t, int32_t total_tokens, int32_t num_groups, int32_t num_q_heads,
                                  int32_t num_kv_heads) {
    const size_t rows = (size_t)prefix_cut_rows(total_tokens, num_groups, num_q_heads, num_kv_heads).slots * kRows;
    const size_t tc = (size_t)prefix_cut_tc(total_tokens, num_groups, num_q_heads, num_kv_heads).slots * kPrefixTcRows;
    return prefix_slots_at(num_groups) + (size_t)prefix_slot_floats(1) * sizeof(float) * (dtype == KDA_BF16 && tc > rows ? tc : rows);
}

cudaError_t launch_prefix_attention(const PrefixAttentionArgs &a, cudaStream_t stream) {
    if (a.cache.total_tokens == 0) return cudaSuccess;
    // The tensor-core kernels keep their running maximum on unscaled scores, in the order that a
    // positive scale leaves alone; any other scale (and fp32) runs on the FMA units.
    const bool tensor = a.dtype == KDA_BF16 && a.scale > 0.f && a.scale <= FLT_MAX;
    return tensor ? launch_prefix_tc(a, stream) : launch_prefix_rows(a, stream);
}

}  // namespace kda
