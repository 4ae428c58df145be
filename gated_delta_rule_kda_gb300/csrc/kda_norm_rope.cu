// Queries and keys normed per head and rotated by position, in one pass; k and v into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s) for each rotated pair
//
// HBM-bound: every element is read once and written once, about eight operations each.  A group of
// 16 lanes takes up to kRows head rows of one token and kind (query, key or value), so that the
// token's cosines and sines, the weights and the place in the cache are fetched once for all of
// them, and the rows' loads are in flight together.  A lane holds two pieces of four channels, at
// ca and cb: with half-split pairs the pieces are the two halves of four pairs (channel i and
// i + rotary_dim / 2), with interleaved pairs they are neighbours; either way both channels of a
// pair are in one lane, and the channels that do not rotate fall to the lanes past rotary_dim / 8.
// Measured (30,195 tokens, 96 + 8 + 8 heads, bf16 into the cache, 1.74 GB): 284 us, 6.12 TB/s, 0.90
// of the measured copy bandwidth; with 256-thread blocks 321 us, four rows a group 307, the rows in
// two batches of four 344: the loads in flight set the pace.  (Eight blocks an SM leave 64 registers: the
// instantiations that append spill 36 to 56 bytes.)
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kGroup = 16;  // lanes of a head row

// A piece as it is loaded; head rows of a group, whose loads are all in flight together.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
    using Raw = float4;
    static constexpr int kRows = 4;
};
template <>
struct Piece<__nv_bfloat16> {
    using Raw = uint2;
    static constexpr int kRows = 8;
};
__device__ __forceinline__ float4 widen(float4 r) { return r; }
__device__ __forceinline__ float4 widen(uint2 r) {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float4 mul4(float4 x, float4 y) {
    return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w);
}
__device__ __forceinline__ float dot4(float4 x) { return x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w; }

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
__global__ void __launch_bounds__(kThreads, 8) norm_rope_kernel(const NormRopeArgs a, uint32_t q_chunks, uint32_t kv_chunks) {
    const int lane = threadIdx.x & (kGroup - 1);
    const uint32_t group = blockIdx.x * (kThreads / kGroup) + threadIdx.x / kGroup;
    const uint32_t per_token = q_chunks + (kAppend ? 2 : 1) * kv_chunks;
    const uint32_t token = group / per_token;
    uint32_t chunk = group - token * per_token;
    constexpr int kRows = Piece<Tin>::kRows;
    using Raw = typename Piece<Tin>::Raw;
    const bool in = token < (uint32_t)a.cache.total_tokens;  // the others stay for the shuffles
    const int32_t t = in ? (int32_t)token : 0;
    // the kind of this group's rows: 0 queries, 1 keys, 2 values
    int kind = 0;
    if (chunk >= q_chunks) {
        chunk -= q_chunks;
        kind = chunk >= kv_chunks ? 2 : 1;
        if (kind == 2) chunk -= kv_chunks;
    }
    const int32_t heads = kind == 0 ? a.num_q_heads : a.num_kv_heads, h0 = (int32_t)chunk * kRows;
    const int32_t rows = in ? min(kRows, heads - h0) : 0;

    const int32_t turning = a.rotary_dim / 8;  // lanes with channels to rotate
    const bool rotated = kind != 2 && lane < turning;
    int32_t ca = 8 * lane, cb = 8 * lane + 4;
    if (!kInterleaved && lane < turning) {
        ca = 4 * lane;
        cb = a.rotary_dim / 2 + 4 * lane;
    }
    const Tin *src = static_cast<const Tin *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                     t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (int64_t)h0 * kD;

    grid_wait();
    Raw ra[kRows], rb[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        ra[i] = rb[i] = Raw{};
        if (i < rows) {
            ra[i] = __ldcs(reinterpret_cast<const Raw *>(src + i * kD + ca));
            rb[i] = __ldcs(reinterpret_cast<const Raw *>(src + i * kD + cb));
        }
    }

    float4 cs0 = make_float4(1.f, 0.f, 1.f, 0.f), cs1 = cs0;  // (c, s) of this lane's four pairs
    float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
    bool ok = in;
    if (in && a.rotary_dim > 0) {
        const int32_t pos = a.positions[t];
        ok = (uint32_t)pos < (uint32_t)a.num_positions;
        if (!ok && lane == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)t);
        if (ok && rotated) {
            const float4 *cs = reinterpret_cast<const float4 *>(a.rope_table + ((int64_t)pos * (a.rotary_dim / 2) + 4 * lane) * 2);
            cs0 = cs[0];
            cs1 = cs[1];
        }
    }
    const float *w = kind == 0 ? a.q_weight : a.k_weight;
    const bool norm = a.norm && kind != 2;
    if (norm && w != nullptr) {
        wa = load4(w + ca);
        wb = load4(w + cb);
    }
    Tout *dst;
    int64_t pitch = kD;  // from head to head
    if (kind == 0) {
        dst = static_cast<Tout *>(a.q_out) + ((int64_t)t * a.num_q_heads + h0) * kD;
    } else if (!kAppend) {
        dst = static_cast<Tout *>(a.k_out) + ((int64_t)t * a.num_kv_heads + h0) * kD;
    } else {
        const Place place = in ? place_of(a.cache, t) : Place{-1, 0};
        if (in && place.page < 0) {
            ok = false;
            if (lane == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)t);
        }
        pitch = (int64_t)a.cache.page_size * kD;
        dst = static_cast<Tout *>(a.kv_pool) + (((int64_t)max(place.page, 0) * 2 + kind - 1) * a.num_kv_heads + h0) * pitch +
              (int64_t)place.at * kD;
    }

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float4 xa = widen(ra[i]), xb = widen(rb[i]);
        float inv = 1.f;
        if (a.norm) {  // a kernel argument: the same for every lane
            float ss = dot4(xa) + dot4(xb);
#pragma unroll
            for (int off = kGroup / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (norm) inv = rsqrtf(ss * (1.f / kD) + a.eps);
        }
        if (kind != 2) {
            const float4 u = mul4(mul4(xa, make_float4(inv, inv, inv, inv)), wa);
            const float4 v = mul4(mul4(xb, make_float4(inv, inv, inv, inv)), wb);
            if (!rotated) {  // 1 and 0 in place of c and s would turn an infinity into NaN
                xa = u;
                xb = v;
            } else if (kInterleaved) {
                xa = make_float4(u.x * cs0.x - u.y * cs0.y, u.y * cs0.x + u.x * cs0.y, u.z * cs0.z - u.w * cs0.w,
                                 u.w * cs0.z + u.z * cs0.w);
                xb = make_float4(v.x * cs1.x - v.y * cs1.y, v.y * cs1.x + v.x * cs1.y, v.z * cs1.z - v.w * cs1.w,
                                 v.w * cs1.z + v.z * cs1.w);
            } else {
                xa = make_float4(u.x * cs0.x - v.x * cs0.y, u.y * cs0.z - v.y * cs0.w, u.z * cs1.x - v.z * cs1.y,
                                 u.w * cs1.z - v.w * cs1.w);
                xb = make_float4(v.x * cs0.x + u.x * cs0.y, v.y * cs0.z + u.y * cs0.w, v.z * cs1.x + u.z * cs1.y,
                                 v.w * cs1.z + u.w * cs1.w);
            }
        }
        if (ok && i < rows) {
            store4(dst + i * pitch + ca, xa);
            store4(dst + i * pitch + cb, xb);
        }
    }
}

template <typename Tin, typename Tout, bool kAppend>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream) {
    constexpr int kRows = Piece<Tin>::kRows;
    const uint32_t q_chunks = (a.num_q_heads + kRows - 1) / kRows, kv_chunks = (a.num_kv_heads + kRows - 1) / kRows;
    const int64_t groups = (int64_t)a.cache.total_tokens * (q_chunks + (kAppend ? 2 : 1) * kv_chunks);
    const unsigned grid = (unsigned)((groups + kThreads / kGroup - 1) / (kThreads / kGroup));
    const auto kernel = a.interleaved ? norm_rope_kernel<Tin, Tout, kAppend, true> : norm_rope_kernel<Tin, Tout, kAppend, false>;
    return launch_serial(kernel, dim3(grid), kThreads, 0, stream, a, q_chunks, kv_chunks);
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
