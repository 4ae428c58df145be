// Attention of 32 rows over tiles of 64 keys in fp32 on the FMA units, by 128 threads: what
// kda_window_attention and kda_prefix_attention share.
//
//   s = scale q k^T;  m' = max(m, max s);  l <- l e^(m - m') + sum e^(s - m');
//   o <- o e^(m - m') + e^(s - m') v
// Tiles of q, k, v and of the probabilities lie in shared memory as fp32; a thread computes 4 x 4
// scores and 4 x 8 outputs, so that each shared-memory read feeds two to four FMAs.  A key that a
// row does not see takes no part: its score is replaced (never computed with), its probability of
// zero skips the product with v, and keys past the end or without a page are loaded as zeros.
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace rows {

constexpr int kThreads = 128;
constexpr int kRows = 32;              // of an item
constexpr int kTile = 64;              // keys of a tile
constexpr int kWarps = kThreads / 32;
constexpr int kPitch = kD + 4;         // q, k rows: float4 reads of 16 rows hit distinct banks
constexpr int kPitchP = kTile + 4;
constexpr size_t kSmem = sizeof(float) * ((kRows + kTile) * kPitch + kTile * kD + kRows * kPitchP);  // two CTAs an SM

struct Tiles {
    float *q, *k, *v, *p;  // [32][kPitch], [64][kPitch], [64][128], [32][kPitchP]
    __device__ __forceinline__ explicit Tiles(float4 *smem) {
        q = reinterpret_cast<float *>(smem);
        k = q + kRows * kPitch;
        v = k + kTile * kPitch;
        p = v + kTile * kD;
    }
};
struct Keys {
    int64_t at[kTile];   // the tile's keys as rows of the pool, or -1
    uint32_t mapped[2];  // bit j: key j of the tile has a page
};

// What a thread (tx = tid % 16, ty = tid / 16) holds of rows 4 ty + i: channels 4 tx .. and 64 + 4 tx ..
struct State {
    float o[4][8], m[4], l[4];
    __device__ __forceinline__ State() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) o[i][c] = 0.f;
        }
    }
};

// Rows of q, a warp a row of 128 channels: source(row) is where row `row` of the 32 starts, or null.
template <typename Source>
__device__ __forceinline__ void load_q(const Tiles &t, Source source) {
    const int warp = threadIdx.x >> 5, c4 = (threadIdx.x & 31) * 4;
    float4 x[kRows / kWarps];
#pragma unroll
    for (int i = 0; i < kRows / kWarps; ++i) {
        const auto *src = source(warp + kWarps * i);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src != nullptr) x[i] = load4(src + c4);
    }
#pragma unroll
    for (int i = 0; i < kRows / kWarps; ++i) *reinterpret_cast<float4 *>(t.q + (warp + kWarps * i) * kPitch + c4) = x[i];
}

// One tile of keys [j0, j0 + 64) of kv head h in a row of the table, none of them from `end` on
// (end <= table_width * page_size).  seen(i, j): whether row 4 ty + i sees key j, if it is mapped.
template <typename T, typename Seen>
__device__ __forceinline__ void tile(const Tiles &t, Keys &keys, State &st, const T *pool, const CacheArgs &cache,
                                     int32_t num_kv_heads, int32_t h, int32_t table_row, int32_t j0, int32_t end,
                                     float scale, Seen seen) {
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, c4 = (tid & 31) * 4;
    auto &o = st.o;
    auto &m = st.m;
    auto &l = st.l;
    __syncthreads();  // the previous tile has been used
    if (tid < kTile) {  // where the tile's keys lie, and which of them exist
        const int32_t j = j0 + tid;
        int64_t at = -1;
        if (j < end) {
            const int32_t page = cache.page_table[(int64_t)table_row * cache.table_width + j / cache.page_size];
            if ((uint32_t)page < (uint32_t)cache.num_pages)
                at = ((int64_t)page * 2 * num_kv_heads + h) * cache.page_size + j % cache.page_size;
        }
        keys.at[tid] = at;
        const uint32_t exist = __ballot_sync(0xffffffffu, at >= 0);
        if ((tid & 31) == 0) keys.mapped[warp] = exist;
    }
    __syncthreads();
    const int64_t kv_stride = (int64_t)num_kv_heads * cache.page_size * kD;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float4 x[kTile / kWarps];
#pragma unroll
        for (int i = 0; i < kTile / kWarps; ++i) {
            const int64_t at = keys.at[warp + kWarps * i];
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at >= 0) x[i] = load4(pool + at * kD + kv * kv_stride + c4);
        }
#pragma unroll
        for (int i = 0; i < kTile / kWarps; ++i)
            *reinterpret_cast<float4 *>(kv ? t.v + (warp + kWarps * i) * kD + c4 : t.k + (warp + kWarps * i) * kPitch + c4) = x[i];
    }
    __syncthreads();
    const uint64_t mapped = (uint64_t)keys.mapped[1] << 32 | keys.mapped[0];

    float s[4][4];  // rows 4 ty + i, keys tx + 16 j
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < kD; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(t.q + (4 * ty + i) * kPitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(t.k + (tx + 16 * j) * kPitch + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = tx + 16 * j;
            const bool sees = seen(i, j0 + k) && (mapped >> k & 1);
            s[i][j] = sees ? s[i][j] * scale : -INFINITY;
            top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float base = top == -INFINITY ? 0.f : top;  // nothing visible yet: e^-inf = 0
        const float keep = expf(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float e = expf(s[i][j] - base);
            t.p[(4 * ty + i) * kPitchP + tx + 16 * j] = e;
            sum += e;
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        m[i] = top;
        l[i] = fmaf(l[i], keep, sum);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[i][c] *= keep;
    }
    __syncwarp();  // a row's probabilities are written and read by the same half-warp
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        float4 e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = *reinterpret_cast<const float4 *>(t.p + (4 * ty + i) * kPitchP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const float4 v0 = *reinterpret_cast<const float4 *>(t.v + (k + kk) * kD + 4 * tx);
            const float4 v1 = *reinterpret_cast<const float4 *>(t.v + (k + kk) * kD + 64 + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = kk == 0 ? e[i].x : kk == 1 ? e[i].y : kk == 2 ? e[i].z : e[i].w;
                if (w != 0.f) {  // NaN counts as well
                    o[i][0] = fmaf(w, v0.x, o[i][0]); o[i][1] = fmaf(w, v0.y, o[i][1]);
                    o[i][2] = fmaf(w, v0.z, o[i][2]); o[i][3] = fmaf(w, v0.w, o[i][3]);
                    o[i][4] = fmaf(w, v1.x, o[i][4]); o[i][5] = fmaf(w, v1.y, o[i][5]);
                    o[i][6] = fmaf(w, v1.z, o[i][6]); o[i][7] = fmaf(w, v1.w, o[i][7]);
                }
            }
        }
    }
}

}  // namespace rows
}  // namespace kda
