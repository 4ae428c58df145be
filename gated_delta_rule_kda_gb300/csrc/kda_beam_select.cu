// The best continuations of a batch of beams.
//
//   total(k, v) = score[k] + x[v] - lse_k,  lse_k = M + log sum_u e^(x[u] - M)
// Within a beam the order of the totals is that of the logits, so the first launch reads each logit
// once and leaves, for every segment of a row, its maximum, its sum of e^(x - max) and its N best
// logits in falling order; the second joins a prompt's K x S lists: log-sum-exp in 64 bits, then the
// list with the best head gives one continuation after the other.
//
// A CTA holds its segment in registers.  Its candidates are found with a bound: threads are taken in
// groups, as many as N or more, and the smallest of the groups' maxima has at least N logits at or
// above it (g groups of random logits: about g ln g).  What reaches the bound is ranked by counting.
// Where too much does (few distinct values, a mask of the lowest value, a short segment) the CTA takes
// its best logits one by one.
// Bound: reading the logits once.
#include "kda_common.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kFound = 512;  // candidates that are ranked by counting
constexpr int kMaxN = KDA_MAX_BEAMS;

// A segment's result: max (fp32), sum (fp32), then N keys, best first; 0: no logit.
// A key orders by logit, then by lower token: ordered(x) << 32 | ~token.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t token) {
    return (uint64_t)ordered(x + 0.f) << 32 | (uint32_t)~token;  // (-0 counts as 0)
}
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }

struct Layout {
    int32_t segments, length;  // of a row; logits of a segment
};
__host__ __device__ inline size_t segment_words(int32_t N) { return 1 + (size_t)N; }  // of 8 bytes

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
};

__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
    return (uint64_t)hi << 32 | lo;
}

// kVecs 16-byte vectors a thread.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads) beam_segments_kernel(const BeamSelectArgs a, const Layout lay) {
    constexpr int kN = Vec<T>::n, kEach = kVecs * kN;
    __shared__ float s_max[kThreads / 32], s_sum[kThreads / 32];
    __shared__ float s_group[64];
    __shared__ uint64_t s_found[kFound];
    __shared__ uint64_t s_best[2][kThreads / 32];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t N = a.choices, row = blockIdx.x, seg = blockIdx.y;
    grid_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.ended != nullptr && a.ended[row] != 0) return;  // its logits are not read
    uint64_t *out = static_cast<uint64_t *>(a.workspace) + ((int64_t)row * lay.segments + seg) * segment_words(N);
    const int32_t v0 = seg * lay.length, count = min(lay.length, a.vocab - v0);
    const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride + v0;
    // A thread's logits are [kN k, kN k + kN) of the segment for k = tid, tid + 256, ..., wherever the row starts,
    // so that rows with the same logits have the same sums: a row off a 16-byte boundary is read in
    // 16-byte vectors all the same, and each thread shifts its own and its neighbour's together.
    const int32_t off = (int32_t)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const auto vector = [&](int32_t k) {  // logits [kN k - off, kN k - off + kN); those outside [0, count) are not read
        const int32_t e0 = k * kN - off;
        if (e0 >= 0 && e0 + kN <= count) return __ldcs(reinterpret_cast<const uint4 *>(src - off) + k);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kN; ++e)
            if (e0 + e >= 0 && e0 + e < count) w[e * sizeof(T) / 4] |= bits(src[e0 + e]) << (e * sizeof(T) % 4 * 8);
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    uint4 raw[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = vector(i * kThreads + tid);
    if (off != 0) {
        const uint32_t shift = off * sizeof(T) * 8;  // bits
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint4 next;
            next.x = __shfl_down_sync(0xffffffffu, raw[i].x, 1);
            next.y = __shfl_down_sync(0xffffffffu, raw[i].y, 1);
            next.z = __shfl_down_sync(0xffffffffu, raw[i].z, 1);
            next.w = __shfl_down_sync(0xffffffffu, raw[i].w, 1);
            if (lane == 31) next = vector(i * kThreads + tid + 1);
            uint32_t w[8] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w, next.x, next.y, next.z, next.w};
            if (shift & 64) {
#pragma unroll
                for (int e = 0; e < 6; ++e) w[e] = w[e + 2];
            }
            if (shift & 32) {
#pragma unroll
                for (int e = 0; e < 5; ++e) w[e] = w[e + 1];
            }
            raw[i].x = __funnelshift_r(w[0], w[1], shift & 31);
            raw[i].y = __funnelshift_r(w[1], w[2], shift & 31);
            raw[i].z = __funnelshift_r(w[2], w[3], shift & 31);
            raw[i].w = __funnelshift_r(w[3], w[4], shift & 31);
        }
    }
    float x[kEach];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        const int32_t left = count - (i * kThreads + tid) * kN;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            if (kN == 4) x[i * kN + e] = __uint_as_float(w[e & 3]);
            else x[i * kN + e] = __uint_as_float(e & 1 ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
            if (e >= left) x[i * kN + e] = -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        x[i] = clean(x[i]);
        top = fmaxf(top, x[i]);
    }
    // the maxima of the groups of threads (32, 16, 8 or 4 of them), and of all
    const int group = N <= 8 ? 32 : N <= 16 ? 16 : N <= 32 ? 8 : 4;
    float g = top;
    for (int o = 1; o < group; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (lane % group == 0) s_group[tid / group] = g;
    float m = g;
    for (int o = group; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_max[warp] = m;
    if (tid == 0) s_count = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, s_max[w]);
    float bound = INFINITY;
    for (int i = lane; i < kThreads / group; i += 32) bound = fminf(bound, s_group[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bound = fminf(bound, __shfl_xor_sync(0xffffffffu, bound, o));
    const float shift = m == -INFINITY ? 0.f : m;
    constexpr float kLog2e = 1.4426950408889634f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += tc::ex2_approx((x[i] - shift) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    if (top >= bound) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float y = x[i * kN + e];
                if (y >= bound && y > -INFINITY) {
                    const int at = atomicAdd(&s_count, 1);
                    if (at < kFound) s_found[at] = make_key(y, (uint32_t)(v0 + (i * kThreads + tid) * kN + e));
                }
            }
    }
    __syncthreads();
    if (tid == 0) {
        sum = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) sum += s_sum[w];
        out[0] = (uint64_t)__float_as_uint(sum) << 32 | __float_as_uint(m);
    }
    const int found = s_count;
    if (found <= kFound) {
        for (int i = tid; i < max(found, N); i += kThreads) {
            if (i >= found) {  // fewer than N logits
                out[1 + i] = 0;
                continue;
            }
            const uint64_t key = s_found[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += s_found[j] > key;
            if (rank < N) out[1 + rank] = key;
        }
        return;
    }
    // One by one: each thread's best logit below the last one taken.
    uint64_t last = ~0ull, mine = 0;
    bool stale = true;
    for (int n = 0; n < N; ++n) {
        if (stale) {
            mine = 0;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const float y = x[i * kN + e];
                    const uint64_t key = make_key(y, (uint32_t)(v0 + (i * kThreads + tid) * kN + e));
                    if (y > -INFINITY && key < last && key > mine) mine = key;
                }
            stale = false;
        }
        const uint64_t best = warp_max(mine);
        if (lane == 0) s_best[n & 1][warp] = best;
        __syncthreads();
        uint64_t all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) all = max(all, s_best[n & 1][w]);
        if (tid == 0) out[1 + n] = all;
        if (mine == all) {  // (0: none is left, anywhere)
            last = all;
            stale = all != 0;
        }
    }
}

// A total as a number that orders the same way (of -inf and below: 0).
__device__ __forceinline__ uint64_t ordered64(double x) {
    if (!(x > -INFINITY)) return 0;
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered64(uint64_t o) {
    return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}

// A warp a prompt.  Lane l owns the lists l, l + 32, ...: list i is segment i % S of beam i / S.
__global__ void __launch_bounds__(32) beam_join_kernel(const BeamSelectArgs a, const Layout lay) {
    constexpr uint32_t kAll = 0xffffffffu;
    __shared__ double s_score[KDA_MAX_BEAMS], s_lse[KDA_MAX_BEAMS];
    extern __shared__ uint8_t s_next[];       // of each list: its next key
    const int lane = threadIdx.x;
    const int32_t b = blockIdx.x, K = a.beams, N = a.choices, S = lay.segments, lists = K * S;
    grid_wait();
    const uint64_t *keys = static_cast<const uint64_t *>(a.workspace) + (int64_t)b * lists * segment_words(N);
    uint64_t over = 0;  // bit k: beam k has ended
    for (int32_t k = 0; k < K; ++k) {
        const float score = a.scores[b * K + k];
        const double s = score != score ? -INFINITY : (double)score;
        const bool end = a.ended != nullptr && a.ended[b * K + k] != 0;
        if (lane == 0) s_score[k] = s;
        if (end) {
            over |= 1ull << k;
            continue;
        }
        float m = -INFINITY;
        for (int32_t i = lane; i < S; i += 32) m = fmaxf(m, __uint_as_float((uint32_t)keys[(int64_t)(k * S + i) * segment_words(N)]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        double sum = 0;
        for (int32_t i = lane; i < S; i += 32) {
            const uint64_t w = keys[(int64_t)(k * S + i) * segment_words(N)];
            const float mi = __uint_as_float((uint32_t)w);
            if (mi > -INFINITY) sum += (double)__uint_as_float((uint32_t)(w >> 32)) * exp((double)mi - (double)m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) s_lse[k] = (double)m + log(sum);  // (without logits there are no keys)
    }
    for (int32_t i = lane; i < lists; i += 32) s_next[i] = 0;
    __syncwarp();
    // the head of list i: (total as an ordered number, key)
    const auto head = [&](int32_t i, uint64_t &total, uint64_t &key) {
        const int32_t k = i / S, n = s_next[i];
        total = 0;
        key = 0;
        if (over >> k & 1) {
            if (i % S != 0 || n > 0) return;
            key = make_key(0.f, (uint32_t)a.end_token);
            total = ordered64(s_score[k]);
        } else if (n < N) {
            key = keys[(int64_t)i * segment_words(N) + 1 + n];
            if (key != 0) total = ordered64(s_score[k] + ((double)unordered((uint32_t)(key >> 32)) - s_lse[k]));
        }
    };
    // The lane's best list: higher total, then lower beam, then higher key.
    uint64_t best = 0, best_key = 0;
    int32_t best_list = -1;
    const auto look = [&] {
        best = best_key = 0;
        best_list = -1;
        for (int32_t i = lane; i < lists; i += 32) {
            uint64_t t, key;
            head(i, t, key);
            if (t > best || (t == best && t != 0 && i / S == best_list / S && key > best_key)) {
                best = t;
                best_key = key;
                best_list = i;
            }
        }
    };
    look();
    for (int32_t n = 0; n < N; ++n) {
        const uint64_t top = warp_max(best);
        const int64_t at = (int64_t)b * N + n;
        if (top == 0) {
            if (lane == 0) {
                a.parent[at] = a.token[at] = -1;
                a.score[at] = -INFINITY;
                if (a.ended_out != nullptr) a.ended_out[at] = 0;
            }
            continue;
        }
        const uint32_t k = __reduce_min_sync(kAll, best == top ? (uint32_t)(best_list / S) : 0xffffffffu);
        const bool mine = best == top && (uint32_t)(best_list / S) == k;
        const uint64_t key = warp_max(mine ? best_key : 0);
        if (mine && best_key == key) {  // keys differ within a beam
            const int32_t token = (int32_t)~(uint32_t)key;
            a.parent[at] = (int32_t)k;
            a.token[at] = token;
            a.score[at] = (float)unordered64(top);
            if (a.ended_out != nullptr) a.ended_out[at] = (over >> k & 1) || token == a.end_token;
            ++s_next[best_list];
            look();
        }
        __syncwarp();
    }
}

Layout layout(kda_dtype dtype, int32_t vocab, int vecs) {
    const int32_t length = kThreads * vecs * (dtype == KDA_BF16 ? 8 : 4);
    return Layout{(vocab + length - 1) / length, length};
}

template <typename T, int kVecs>
cudaError_t launch(const BeamSelectArgs &a, const Layout &lay, cudaStream_t stream) {
    return launch_serial(beam_segments_kernel<T, kVecs>, dim3((unsigned)(a.batch * a.beams), (unsigned)lay.segments), kThreads,
                         0, stream, a, lay);
}

}  // namespace

size_t beam_select_workspace(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    const Layout lay = layout(KDA_FP32, vocab, 4);  // the most segments of any call
    return (size_t)batch * beams * lay.segments * segment_words(choices) * 8;
}

cudaError_t launch_beam_select(const BeamSelectArgs &a, cudaStream_t stream) {
    const int vecs = 4;
    const Layout lay = layout(a.dtype, a.vocab, vecs);
    const cudaError_t e = a.dtype == KDA_BF16 ? launch<__nv_bfloat16, vecs>(a, lay, stream) : launch<float, vecs>(a, lay, stream);
    if (e != cudaSuccess) return e;
    return launch_serial(beam_join_kernel, dim3((unsigned)a.batch), 32, (size_t)a.beams * lay.segments, stream, a, lay);
}

}  // namespace kda
