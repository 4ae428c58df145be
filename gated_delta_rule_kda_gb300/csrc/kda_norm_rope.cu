// Queries and keys normed per head and rotated by position, in one pass; k and v into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s) for each rotated pair
//
// HBM-bound: every element is read once and written once, about eight operations each.  A group
// of 16 lanes takes kRows head rows of one token, eight channels a lane (16-byte accesses in
// bf16): the sum of squares is four shuffles, and the token's cosines and sines stay in registers
// for the group's rows.  rotary_dim is a multiple of 16, so with half-split pairs channel c of
// lane l meets channel c of one other lane (a shuffle); interleaved pairs lie within a lane.
// The rows of a token are its query heads, its key heads, and with a cache its value heads.
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;  // lanes of a head row
constexpr int kRows = 4;    // head rows of a group
constexpr int kVec = kD / kGroup;

__device__ __forceinline__ void load8(const float *p, float (&x)[kVec]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[kVec]) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[kVec]) {
    store4(p, make_float4(x[0], x[1], x[2], x[3]));
    store4(p + 4, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[kVec]) {
    uint4 r;
    uint32_t *w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = r;
}

// Where the keys of token t go: the page and the place in it, or page -1.
struct Place {
    int32_t page, at;
};
__device__ __forceinline__ Place place_of(const CacheArgs &c, int32_t t) {
    int32_t lo = 0, hi = c.batch;  // the last b in [0, batch) with cu[b] <= t
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (c.cu_tokens[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int32_t first = c.cu_tokens[lo], end = c.cu_tokens[lo + 1], row = c.slot[lo];
    if (t < first || t >= end || (uint32_t)row >= (uint32_t)c.table_rows) return {-1, 0};
    const int32_t len = c.kv_len[row];
    if (len < 0 || len > c.table_width * c.page_size) return {-1, 0};
    const int64_t j = (int64_t)len - end + t;  // below len: t < end
    if (j < 0) return {-1, 0};
    const int32_t page = c.page_table[(int64_t)row * c.table_width + j / c.page_size];
    return {(uint32_t)page < (uint32_t)c.num_pages ? page : -1, (int32_t)(j % c.page_size)};
}

template <typename Tin, typename Tout, bool kAppend, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a, int32_t chunks) {
    const int lane = threadIdx.x & (kGroup - 1);
    const int64_t group = (int64_t)blockIdx.x * (kThreads / kGroup) + threadIdx.x / kGroup;
    const int32_t T = a.cache.total_tokens, Hq = a.num_q_heads, Hkv = a.num_kv_heads;
    const int32_t rows = Hq + (kAppend ? 2 : 1) * Hkv;
    const bool in = group < (int64_t)T * chunks;  // every lane stays for the shuffles
    const int32_t t = in ? (int32_t)(group / chunks) : 0;
    const int32_t r0 = in ? (int32_t)(group % chunks) * kRows : rows;

    float x[kRows][kVec];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int32_t r = r0 + i;
        if (r < rows) {
            const Tin *src = r < Hq ? static_cast<const Tin *>(a.q) + t * a.q_stride + (int64_t)r * kD
                             : r < Hq + Hkv
                                 ? static_cast<const Tin *>(a.k) + t * a.k_stride + (int64_t)(r - Hq) * kD
                                 : static_cast<const Tin *>(a.v) + t * a.v_stride + (int64_t)(r - Hq - Hkv) * kD;
            load8(src + lane * kVec, x[i]);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[i][j] = 0.f;
        }
    }

    // this lane's pairs: cosines and sines of channels 8 lane .. 8 lane + 7
    const int32_t half_lanes = a.rotary_dim / (2 * kVec);  // lanes of the first elements (half-split)
    const bool rotated = lane < 2 * half_lanes;
    float c[kInterleaved ? kVec / 2 : kVec], s[kInterleaved ? kVec / 2 : kVec];
    bool ok = in;
    if (in && a.rotary_dim > 0) {
        const int32_t pos = a.positions[t];
        ok = (uint32_t)pos < (uint32_t)a.num_positions;
        if (!ok && lane == 0 && r0 == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)t);
        if (ok && rotated) {
            constexpr int n = kInterleaved ? kVec / 2 : kVec;
            const int32_t first = kInterleaved ? lane * n : (lane < half_lanes ? lane : lane - half_lanes) * n;
            const float4 *cs = reinterpret_cast<const float4 *>(
                a.rope_table + ((int64_t)pos * (a.rotary_dim / 2) + first) * 2);
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                const float4 y = cs[i];
                c[2 * i] = y.x; s[2 * i] = y.y;
                c[2 * i + 1] = y.z; s[2 * i + 1] = y.w;
            }
        }
    }
    Place place{-1, 0};
    if (kAppend && in && r0 + kRows > Hq) {
        place = place_of(a.cache, t);
        if (place.page < 0 && lane == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)t);
    }

    const int partner = lane < half_lanes ? lane + half_lanes : lane - half_lanes;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int32_t r = r0 + i;
        const bool value = kAppend && r >= Hq + Hkv;
        if (a.norm) {  // a kernel argument: the same for every lane
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < kVec; ++j) ss = fmaf(x[i][j], x[i][j], ss);
#pragma unroll
            for (int off = kGroup / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (!value) {
                const float inv = 1.f / sqrtf(ss * (1.f / kD) + a.eps);
                const float *w = r < Hq ? a.q_weight : a.k_weight;
                if (w != nullptr) {
                    const float4 w0 = load4(w + lane * kVec), w1 = load4(w + lane * kVec + 4);
                    const float wv[kVec] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int j = 0; j < kVec; ++j) x[i][j] = x[i][j] * inv * wv[j];
                } else {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) x[i][j] *= inv;
                }
            }
        }
        if (kInterleaved) {
            if (rotated && !value) {
#pragma unroll
                for (int j = 0; j < kVec / 2; ++j) {
                    const float u = x[i][2 * j], v = x[i][2 * j + 1];
                    x[i][2 * j] = u * c[j] - v * s[j];
                    x[i][2 * j + 1] = v * c[j] + u * s[j];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float other = __shfl_sync(0xffffffffu, x[i][j], partner & (kGroup - 1), kGroup);
                if (rotated && !value)
                    x[i][j] = lane < half_lanes ? x[i][j] * c[j] - other * s[j] : x[i][j] * c[j] + other * s[j];
            }
        }
        if (!ok || r >= rows) continue;  // no shuffle of this row is left
        Tout *dst;
        if (r < Hq) {
            dst = static_cast<Tout *>(a.q_out) + ((int64_t)t * Hq + r) * kD;
        } else if (kAppend) {
            if (place.page < 0) continue;
            const int32_t kv = value ? 1 : 0, h = r - Hq - kv * Hkv;
            dst = static_cast<Tout *>(a.kv_pool) +
                  ((((int64_t)place.page * 2 + kv) * Hkv + h) * a.cache.page_size + place.at) * kD;
        } else {
            dst = static_cast<Tout *>(a.k_out) + ((int64_t)t * Hkv + (r - Hq)) * kD;
        }
        store8(dst + lane * kVec, x[i]);
    }
}

template <typename Tin, typename Tout, bool kAppend>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream) {
    const int32_t rows = a.num_q_heads + (kAppend ? 2 : 1) * a.num_kv_heads;
    const int32_t chunks = (rows + kRows - 1) / kRows;
    const int64_t groups = (int64_t)a.cache.total_tokens * chunks;
    const unsigned grid = (unsigned)((groups + kThreads / kGroup - 1) / (kThreads / kGroup));
    if (a.interleaved) norm_rope_kernel<Tin, Tout, kAppend, true><<<grid, kThreads, 0, stream>>>(a, chunks);
    else norm_rope_kernel<Tin, Tout, kAppend, false><<<grid, kThreads, 0, stream>>>(a, chunks);
    return cudaGetLastError();
}
template <typename Tin, typename Tout>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream) {
    return a.kv_pool != nullptr ? launch<Tin, Tout, true>(a, stream) : launch<Tin, Tout, false>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs &a, cudaStream_t stream) {
    if (a.cache.total_tokens == 0) return cudaSuccess;
    if (a.in_dtype == KDA_BF16)
        return a.out_dtype == KDA_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                       : launch<__nv_bfloat16, float>(a, stream);
    return a.out_dtype == KDA_BF16 ? launch<float, __nv_bfloat16>(a, stream) : launch<float, float>(a, stream);
}

}  // namespace kda
