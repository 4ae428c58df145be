// The best continuations of a batch of beams.
//
//   total(k, v) = score[k] + x[v] - lse_k,  lse_k = M + log sum_u e^(x[u] - M)
// Within a beam the order of the totals is that of the logits, so the first launch reads each logit
// once and leaves, for every segment of a row, its maximum, its sum of e^(x - max) and its N best
// logits in falling order; the second joins a prompt's K x S lists: log-sum-exp in 64 bits, then the
// list with the best head gives one continuation after the other.
//
// A CTA goes over its segment in chunks.  Candidates are found with a bound from the first one: threads are taken
// in groups, more than N, and the N-th best of the groups' maxima has at least N logits at or above it, and few
// more.  What reaches the bound, in any chunk, is kept and ranked by counting.
// Where too much does, the logits are gone through once more with the bound of all of them, and where that
// leaves too much as well (few distinct values, a mask of the lowest value, a short segment) the CTA takes its
// best logits one by one.
// Bound: reading the logits once.
#include "kda_common.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kFound = 512;  // candidates that are ranked by counting
constexpr int kHeld = 384;   // vectors with a candidate that a CTA holds
constexpr int kCtasSm = 6;
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

struct Layout {
    int32_t segments, length;  // of a row; logits of a segment
};
__host__ __device__ inline size_t segment_words(int32_t N) { return 1 + (size_t)N; }  // of 8 bytes

// 16-byte vectors of logits: kN of them.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static constexpr uint32_t kNone = 0xff800000u;  // -inf in each place
    static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float get(const uint32_t *w, int e) { return __uint_as_float(w[e]); }
    // Logit e of a vector in shared memory.
    static __device__ __forceinline__ float at(const uint4 &v, int e) { return reinterpret_cast<const float *>(&v)[e]; }
    // NaN to -inf, +inf to the largest number
    static __device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }
    template <int kVecs = 1>
    static __device__ __forceinline__ float max_of(const uint4 *v) {  // of those that are not NaN (-inf: of none)
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)), fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
        return m;
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
    static __device__ __forceinline__ float get(const uint32_t *w, int e) {
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
    static __device__ __forceinline__ float at(const uint4 &v, int e) {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(&v)[e]);
    }
    static __device__ __forceinline__ float clean(float x) { return Vec<float>::clean(x); }
    template <int kVecs = 1>
    static __device__ __forceinline__ float max_of(const uint4 *v) {
        const auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
        __nv_bfloat162 m = __hmax2(__hmax2(two(v[0].x), two(v[0].y)), __hmax2(two(v[0].z), two(v[0].w)));
#pragma unroll
        for (int i = 1; i < kVecs; ++i)
            m = __hmax2(m, __hmax2(__hmax2(two(v[i].x), two(v[i].y)), __hmax2(two(v[i].z), two(v[i].w))));
        return fmaxf(-INFINITY, fmaxf(__low2float(m), __high2float(m)));
    }
};

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
    return (uint64_t)hi << 32 | lo;
}

// Logits [e0, e0 + kN) of a segment at src, -inf in place of those outside [0, count), which are not read.
template <typename T>
__device__ __noinline__ uint4 edge_vector(const T *src, int32_t e0, int32_t count) {
    using V = Vec<T>;
    constexpr int kPer = 4 / sizeof(T);
    uint32_t w[4] = {V::kNone, V::kNone, V::kNone, V::kNone};
#pragma unroll
    for (int e = 0; e < V::n; ++e)
        if (e0 + e >= 0 && e0 + e < count) {
            const int at = e / kPer, sh = e % kPer * 16;
            w[at] = (kPer == 1 ? 0u : w[at] & ~(0xffffu << sh)) | V::bits(src[e0 + e]) << sh;
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA goes over its segment in chunks of kVecs 16-byte vectors a thread, each loaded when the last one is done with
// (other CTAs of the SM have loads in flight meanwhile: with a second buffer there were four of them instead of six, and
// 64 x 8 rows of 131,072 took 45 us instead of 38), and no barrier but those of the bound after the first.  What is rare
// is kept out of the loop's code, rolled, and reads from shared memory: unrolled beside it, the instructions did not
// come fast enough (68 us where these take 31, 512 rows of 131,072 bf16 logits: 4.3 TB/s).
template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads, kCtasSm) beam_segments_kernel(const BeamSelectArgs a, const Layout lay) {
    using V = Vec<T>;
    constexpr int kN = V::n, kChunk = kThreads * kVecs * kN;
    constexpr float kMost = 3.402823466e38f, kLog2e = 1.4426950408889634f;
    constexpr uint32_t kAll = 0xffffffffu;
    __shared__ uint4 s_chunk[kVecs][kThreads];  // places of each thread's own, and a chunk that is taken one by one
    __shared__ uint64_t s_found[kFound], s_kept[kMaxN], s_best[2][kThreads / 32];
    __shared__ float2 s_sum[kThreads / 32];
    __shared__ uint4 s_vector[kHeld];  // vectors that hold a candidate
    __shared__ uint32_t s_token[kHeld];  // and their first token
    __shared__ float s_top[kThreads], s_bound;
    __shared__ int s_held, s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t N = a.choices, row = blockIdx.x, seg = blockIdx.y;
    if (tid == 0) s_count = s_held = 0;
    grid_wait();
    if (a.ended != nullptr && a.ended[row] != 0) return;  // its logits are not read
    uint64_t *out = static_cast<uint64_t *>(a.workspace) + ((int64_t)row * lay.segments + seg) * segment_words(N);
    const int32_t v0 = seg * lay.length, count = min(lay.length, a.vocab - v0), chunks = (count + kChunk - 1) / kChunk;
    const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride + v0;
    // A thread's logits are [kN k, kN k + kN) of the segment for k = tid, tid + 256, ..., wherever the row starts,
    // so that rows with the same logits have the same sums: a row off a 16-byte boundary is read in
    // 16-byte vectors all the same, and each thread shifts its own and its neighbour's together.
    const int32_t off = (int32_t)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const auto vector = [&](int32_t k) {
        const int32_t e0 = k * kN - off;
        return e0 >= 0 && e0 + kN <= count ? __ldcs(reinterpret_cast<const uint4 *>(src - off) + k) : edge_vector(src, e0, count);
    };
    const auto fetch = [&](uint4 (&raw)[kVecs], int32_t c) {
        if ((c > 0 || off == 0) && (c + 1) * kChunk <= count) {  // whole vectors
            const uint4 *at = reinterpret_cast<const uint4 *>(src - off) + c * (kVecs * kThreads) + tid;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) raw[i] = __ldcs(at + i * kThreads);
        } else {
#pragma unroll 1
            for (int i = 0; i < kVecs; ++i) s_chunk[i][tid] = vector((c * kVecs + i) * kThreads + tid);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) raw[i] = s_chunk[i][tid];
        }
    };
    const auto align = [&](uint4 (&raw)[kVecs], int32_t c) {
        const uint32_t shift = off * sizeof(T) * 8;  // bits
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint4 next;
            next.x = __shfl_down_sync(kAll, raw[i].x, 1);
            next.y = __shfl_down_sync(kAll, raw[i].y, 1);
            next.z = __shfl_down_sync(kAll, raw[i].z, 1);
            next.w = __shfl_down_sync(kAll, raw[i].w, 1);
            if (lane == 31) next = vector((c * kVecs + i) * kThreads + tid + 1);
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
    };
    const auto token = [&](int32_t c, int e) {  // of this thread's logit e of chunk c
        return (uint32_t)(v0 + ((c * kVecs + e / kN) * kThreads + tid) * kN + e % kN);
    };
    // The best N of `found` keys, in order, to dst.
    const auto rank = [&](int found, uint64_t *dst) {
        for (int i = tid; i < found; i += kThreads) {
            const uint64_t key = s_found[i];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < found; ++j) r += s_found[j] > key;
            if (r < N) dst[r] = key;
        }
    };

    uint4 raw[kVecs];
    float m = -INFINITY, sum = 0.f;  // of this thread's logits: the maximum, and the sum of e^(x - m)
    float bound = -INFINITY;
    for (int32_t c = 0; c < chunks; ++c) {
        fetch(raw, c);
        if (off != 0) align(raw, c);
        const float top = V::template max_of<kVecs>(raw);
        if (c == 0) {
            // the N-th best of the maxima of 64 groups of threads (N > 32: of the threads), by counting: N logits lie
            // at or above it, and few more
            const int groups = N <= 32 ? 64 : kThreads;
            float g = top;
            for (int o = 1; o < kThreads / groups; o <<= 1) g = fmaxf(g, __shfl_xor_sync(kAll, g, o));
            if (tid % (kThreads / groups) == 0) s_top[tid / (kThreads / groups)] = g;
            __syncthreads();
            if (tid < groups) {
                g = s_top[tid];
                int r = 0;
#pragma unroll 16
                for (int i = 0; i < groups; ++i) r += s_top[i] > g || (s_top[i] == g && i < tid);
                if (r == N - 1) s_bound = g;
            }
            __syncthreads();
            bound = fminf(s_bound, kMost);  // (+inf counts as the largest number, which may come before it)
        }
        // What can be chosen: logits at or above the bound in the first chunk, above it later (N logits reach the
        // bound already, and go before equal ones).
        const bool equal = c == 0;
        const auto reaches = [&](float y) { return (equal ? y >= bound : y > bound) && y > -INFINITY; };
        if (reaches(top)) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (reaches(V::max_of(raw + i))) {
                    const int at = atomicAdd(&s_held, 1);
                    if (at < kHeld) {
                        s_vector[at] = raw[i];
                        s_token[at] = token(c, i * kN);
                    }
                }
        }
        const float now = fmaxf(m, fminf(top, kMost));
        const float shift = now == -INFINITY ? 0.f : now;
        if (now > m) sum *= tc::ex2_approx((m - shift) * kLog2e);
        m = now;
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
                float2 x = make_float2(V::get(w, e), V::get(w, e + 1));
                x = tc::mul2(tc::fma2(x, make_float2(1.f, 1.f), make_float2(-shift, -shift)), make_float2(kLog2e, kLog2e));
                part = tc::fma2(make_float2(tc::ex2_approx(x.x), tc::ex2_approx(x.y)), make_float2(1.f, 1.f), part);
            }
        }
        float add = part.x + part.y;
        if (!(add <= kMost)) {  // a NaN or +inf among the logits
#pragma unroll
            for (int i = 0; i < kVecs; ++i) s_chunk[i][tid] = raw[i];
            add = 0.f;
#pragma unroll 1
            for (int e = 0; e < kVecs * kN; ++e)
                add += tc::ex2_approx((V::clean(V::at(s_chunk[e / kN][tid], e % kN)) - shift) * kLog2e);
        }
        sum += add;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the warps' maxima and sums
    float all = m;
    for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kAll, all, o));
    sum = m == -INFINITY ? 0.f : sum * tc::ex2_approx((m - all) * kLog2e);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) s_sum[warp] = make_float2(all, sum);
    __syncthreads();
    // The held vectors' logits that reach the bound (above it or not: the N that reached it first are among them).
    const auto expand = [&] {
        const int held = s_held;
        if (held <= kHeld) {
            for (int i = tid; i < held * kN; i += kThreads) {
                const float y = V::at(s_vector[i / kN], i % kN);
                if (!(y >= bound && y > -INFINITY)) continue;
                const int at = atomicAdd(&s_count, 1);
                if (at < kFound) s_found[at] = make_key(V::clean(y), s_token[i / kN] + i % kN);
            }
            __syncthreads();
        }
        return held <= kHeld && s_count <= kFound;
    };
    bool few = expand();
    if (!few) {
        // The first chunk's bound was too low for the others (it may be masked for the most part, or N be large): the N-th
        // best of all threads' maxima, and the logits once more (4 prompts x 32 beams, 64 chosen, a fifth of 243,478
        // tokens masked: 95 us, and 410 one by one).
        __syncthreads();
        s_top[tid] = m;
        if (tid == 0) s_held = s_count = 0;
        __syncthreads();
        int r = 0;
#pragma unroll 16
        for (int i = 0; i < kThreads; ++i) r += s_top[i] > m || (s_top[i] == m && i < tid);
        if (r == N - 1) s_bound = m;
        __syncthreads();
        bound = s_bound;
#pragma unroll 1
        for (int32_t c = 0; c < chunks; ++c) {
            fetch(raw, c);
            if (off != 0) align(raw, c);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const float y = V::max_of(raw + i);
                if (!(y >= bound && y > -INFINITY)) continue;
                const int at = atomicAdd(&s_held, 1);
                if (at < kHeld) {
                    s_vector[at] = raw[i];
                    s_token[at] = token(c, i * kN);
                }
            }
        }
        __syncthreads();
        few = expand();
    }
    int found = s_count;
    if (!few) {
        // Too many: each chunk's best, one by one, beside the best of those before.
        found = 0;
        for (int32_t c = 0; c < chunks; ++c) {
            __syncthreads();
            fetch(raw, c);
            if (off != 0) align(raw, c);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) s_chunk[i][tid] = raw[i];
            const uint64_t least = found == N ? s_found[N - 1] : 0;  // (after a barrier: in order)
            uint64_t below = ~0ull, mine = 0;
            bool stale = true;
            int taken = 0;
            for (; taken < N; ++taken) {
                if (stale) {  // this thread's best logit below the last one taken
                    mine = 0;
#pragma unroll 1
                    for (int e = 0; e < kVecs * kN; ++e) {
                        const float y = V::clean(V::at(s_chunk[e / kN][tid], e % kN));
                        const uint64_t key = make_key(y, token(c, e));
                        if (y > -INFINITY && key < below && key > mine) mine = key;
                    }
                    stale = false;
                }
                const uint64_t best = warp_max(mine);
                if (lane == 0) s_best[taken & 1][warp] = best;
                __syncthreads();
                uint64_t next = 0;
                for (int w = 0; w < kThreads / 32; ++w) next = max(next, s_best[taken & 1][w]);
                if (next <= least) break;  // (0: none is left)
                if (tid == 0) s_found[found + taken] = next;
                if (mine == next) {
                    below = next;
                    stale = true;
                }
            }
            __syncthreads();
            rank(found + taken, s_kept);
            __syncthreads();
            found = min(found + taken, N);
            if (tid < found) s_found[tid] = s_kept[tid];
        }
        __syncthreads();
    }
    rank(found, out + 1);
    for (int i = found + tid; i < N; i += kThreads) out[1 + i] = 0;  // (fewer than N logits)
    if (tid == 0) {
        for (int w = 0; w < kThreads / 32; ++w) all = fmaxf(all, s_sum[w].x);
        sum = 0.f;
        for (int w = 0; w < kThreads / 32; ++w)
            if (s_sum[w].x > -INFINITY) sum = fmaf(s_sum[w].y, tc::ex2_approx((s_sum[w].x - all) * kLog2e), sum);
        out[0] = (uint64_t)__float_as_uint(sum) << 32 | __float_as_uint(all);
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

// A continuation; total 0: there is none.
struct Choice {
    uint64_t total, key;
    int32_t beam;
};
// Whether x comes before y.
__device__ __forceinline__ bool before(const Choice &x, const Choice &y) {
    return x.total > y.total || (x.total == y.total && (x.beam < y.beam || (x.beam == y.beam && x.key > y.key)));
}

// A CTA a prompt.  Thread t owns the lists t, t + 256, ...: list i is segment i % S of beam i / S.
// Bound by the chain of its steps (about 6 us: loads, exponentials and logarithms in 64 bits 3, the two rounds of
// counting 2): 64 prompts of 8 beams 8.7 us, of which 6.5 show behind the segments.
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamSelectArgs a, const Layout lay) {
    __shared__ double s_score[KDA_MAX_BEAMS], s_lse[KDA_MAX_BEAMS];
    __shared__ uint64_t s_group[64], s_total[kThreads], s_key[kThreads];
    __shared__ Choice s_found[kFound], s_best[2][kThreads / 32];
    __shared__ int s_count;
    __shared__ uint32_t s_over[2];
    __shared__ float s_max[KDA_MAX_BEAMS];
    extern __shared__ uint8_t s_next[];  // of each list: its next key (one by one)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = blockIdx.x, K = a.beams, N = a.choices, S = lay.segments, lists = K * S;
    const uint64_t *keys = static_cast<const uint64_t *>(a.workspace) + (int64_t)b * lists * segment_words(N);
    const auto list = [&](int32_t i) { return keys + (int64_t)i * segment_words(N); };
    if (tid < 64) {
        s_group[tid] = 0;
        const float score = tid < K ? a.scores[b * K + tid] : 0.f;
        s_score[tid] = score != score ? -INFINITY : (double)score;
        const uint32_t end = __ballot_sync(0xffffffffu, tid < K && a.ended != nullptr && a.ended[b * K + tid] != 0);
        if (lane == 0) s_over[warp] = end;
    }
    if (tid == 0) s_count = 0;
    grid_wait();
    // A thread takes one of the first `depth` continuations of a list (lists <= 256): number n0 of list i0.
    const int32_t depth = min(N, kThreads / lists), n0 = depth > 0 ? tid % depth : 0, i0 = depth > 0 ? tid / depth : lists;
    const uint64_t key0 = i0 < lists ? list(i0)[1 + n0] : 0;
    __syncthreads();
    const uint64_t over = (uint64_t)s_over[1] << 32 | s_over[0];  // bit k: beam k has ended
    // Log-sum-exp in 64 bits, whose units are few: `width` lanes a beam, so that no lane is idle in short rows; the
    // logarithms of all beams at once.
    const int32_t width = S > 16 ? 32 : S > 8 ? 16 : S > 4 ? 8 : S > 2 ? 4 : S;
    for (int32_t k0 = 0; k0 < K; k0 += kThreads / width) {  // (whole warps go round)
        const int32_t k = k0 + tid / width, l = tid % width;
        const bool live = k < K && !(over >> k & 1);
        const uint64_t first = live && l < S ? list(k * S + l)[0] : 0xff800000u;  // (sum, maximum); none: 0, -inf
        float m = __uint_as_float((uint32_t)first);
        if (live)
            for (int32_t i = l + width; i < S; i += width) m = fmaxf(m, __uint_as_float((uint32_t)list(k * S + i)[0]));
        for (int o = width >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const auto part = [&](uint64_t w) {  // (of a segment without logits: nothing)
            const float mi = __uint_as_float((uint32_t)w), x = __uint_as_float((uint32_t)(w >> 32));
            return mi == m ? (double)x : mi > -INFINITY ? (double)x * exp((double)mi - (double)m) : 0.;
        };
        double sum = part(first);
        if (live)
            for (int32_t i = l + width; i < S; i += width) sum += part(list(k * S + i)[0]);
        for (int o = width >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (live && l == 0) {
            s_max[k] = m;
            s_lse[k] = sum;
        }
    }
    __syncthreads();
    if (tid < K && !(over >> tid & 1)) s_lse[tid] = (double)s_max[tid] + log(s_lse[tid]);  // (without logits there are no keys)
    __syncthreads();
    // Continuation n of list i, whose key is given.
    const auto choice_of = [&](int32_t i, int32_t n, uint64_t key) {
        Choice c{0, 0, i / S};
        if (over >> c.beam & 1) {
            if (i % S != 0 || n > 0) return c;
            c.key = make_key(0.f, (uint32_t)a.end_token);
            c.total = ordered64(s_score[c.beam]);
        } else if (key != 0) {
            c.key = key;
            c.total = ordered64(s_score[c.beam] + ((double)unordered((uint32_t)(key >> 32)) - s_lse[c.beam]));
        }
        return c;
    };
    const auto choice = [&](int32_t i, int32_t n) { return choice_of(i, n, n < N ? list(i)[1 + n] : 0); };
    const auto give = [&](int32_t n, const Choice &c) {
        const int64_t at = (int64_t)b * N + n;
        const int32_t token = (int32_t)~(uint32_t)c.key;
        a.parent[at] = c.total == 0 ? -1 : c.beam;
        a.token[at] = c.total == 0 ? -1 : token;
        a.score[at] = c.total == 0 ? -INFINITY : (float)unordered64(c.total);
        if (a.ended_out != nullptr) a.ended_out[at] = c.total != 0 && ((over >> c.beam & 1) || token == a.end_token);
    };
    // A bound that N continuations reach: the N-th best of the threads' continuations, by counting (which are all there
    // are where depth = N); with more lists than threads, the smallest of the best heads of N or more groups of lists.
    // Then what reaches it, in every list whose head does.
    uint64_t bound = 1;
    if (depth > 0) {
        Choice c{0, 0, 0};
        if (i0 < lists) c = choice_of(i0, n0, key0);
        s_total[tid] = c.total;
        s_key[tid] = c.key;
        __syncthreads();
        // Those of one beam lie together: within it the key decides, between beams the total and then the beam.
        const int taken = lists * depth, begin = min(taken, i0 / S * S * depth), end = min(taken, begin + S * depth);
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < begin; ++j) rank += s_total[j] >= c.total;
#pragma unroll 8
        for (int j = begin; j < end; ++j) rank += s_key[j] > c.key;
#pragma unroll 8
        for (int j = end; j < taken; ++j) rank += s_total[j] > c.total;
        if (depth == N) {
            // (totals of 0 are none: they are left out, and what nothing is left for is filled in)
            const int there = __syncthreads_count(c.total != 0);
            if (c.total != 0 && rank < N) give(rank, c);
            for (int n = there + tid; n < N; n += kThreads) give(n, Choice{0, 0, 0});
            return;
        }
        if (c.total != 0 && rank == N - 1) s_group[0] = c.total;
        __syncthreads();
        bound = max(bound, s_group[0]);
    } else {
        const int32_t groups = N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64;
        for (int32_t i = tid; i < lists; i += kThreads) {
            const uint64_t t = choice(i, 0).total;
            if (t != 0) atomicMax(reinterpret_cast<unsigned long long *>(s_group + i % groups), (unsigned long long)t);
        }
        __syncthreads();
        uint64_t least = ~0ull;
        for (int32_t i = 0; i < groups; ++i) least = min(least, s_group[i]);
        bound = max(bound, least);
    }
    const auto filter = [&] {
        for (int32_t at = tid; at < lists * N; at += kThreads) {
            const int32_t i = at / N, n = at - i * N;
            if ((depth > 0 ? s_total[i * depth] : choice(i, 0).total) < bound) continue;  // (a list falls)
            const Choice c = choice(i, n);
            if (c.total < bound) continue;
            const int to = atomicAdd(&s_count, 1);
            if (to >= kFound) continue;
            s_found[to] = c;
        }
        __syncthreads();
    };
    filter();
    if (s_count > kFound && depth > 0) {
        // A beam is ahead, and much of what its lists have goes before the other lists' heads.  The lists that the bound
        // leaves are few: the N-th best of what the threads see when they go further down those is a higher bound (4
        // prompts x 32 beams, 64 of them chosen, 243,478 tokens: 103 us, and 169 when all are taken one by one).
        __syncthreads();
        if (tid == 0) s_count = 0;
        __syncthreads();
        if (tid < lists && s_total[tid * depth] >= bound) s_key[atomicAdd(&s_count, 1)] = (uint64_t)tid;
        __syncthreads();
        const int32_t left = s_count, deeper = min(N, kThreads / left);  // (left > 0: N continuations reach the bound)
        const int32_t n = tid % deeper, k = tid / deeper;
        const uint64_t total = k < left ? choice((int32_t)s_key[k], n).total : 0;
        uint64_t *s_deep = reinterpret_cast<uint64_t *>(s_found);
        s_deep[tid] = total;
        __syncthreads();
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < kThreads; ++j) rank += s_deep[j] > total || (s_deep[j] == total && j < tid);
        if (total != 0 && rank == N - 1) s_group[0] = total;
        __syncthreads();
        bound = max(bound, s_group[0]);
        if (tid == 0) s_count = 0;
        __syncthreads();
        filter();
    }
    const int found = s_count;
    if (found <= kFound) {
        for (int i = tid; i < max(found, N); i += kThreads) {
            if (i >= found) {
                give(i, Choice{0, 0, 0});
                continue;
            }
            const Choice c = s_found[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < found; ++j) {
                const Choice x = s_found[j];
                const bool same = x.beam == c.beam;
                rank += same ? x.key > c.key : x.total > c.total || (x.total == c.total && x.beam < c.beam);
            }
            if (rank < N) give(rank, c);
        }
        return;
    }
    // One by one: the best of the lists' heads.
    for (int32_t i = tid; i < lists; i += kThreads) s_next[i] = 0;
    Choice mine;
    int32_t from = -1;
    const auto look = [&] {
        mine = Choice{0, 0, 0};
        for (int32_t i = tid; i < lists; i += kThreads) {
            const Choice c = choice(i, s_next[i]);
            if (c.total != 0 && (mine.total == 0 || before(c, mine))) {
                mine = c;
                from = i;
            }
        }
    };
    look();
    for (int32_t n = 0; n < N; ++n) {
        Choice best = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Choice c{__shfl_xor_sync(0xffffffffu, best.total, o), __shfl_xor_sync(0xffffffffu, best.key, o),
                           __shfl_xor_sync(0xffffffffu, best.beam, o)};
            if (before(c, best)) best = c;
        }
        if (lane == 0) s_best[n & 1][warp] = best;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w)
            if (before(s_best[n & 1][w], best)) best = s_best[n & 1][w];
        if (tid == 0) give(n, best);
        if (best.total != 0 && mine.total == best.total && mine.beam == best.beam && mine.key == best.key) {
            ++s_next[from];
            look();
        }
    }
}

constexpr int kVecs = 4;        // 16-byte vectors of a chunk, a thread
constexpr int kMostChunks = 4;  // of a segment
constexpr int kWaves = 5;       // CTAs an SM that short segments are for
constexpr size_t kMostLists = KDA_MAX_BEAMS * ((1 << 21) / (kThreads * kVecs * 4));  // of a prompt

Layout layout(kda_dtype dtype, int32_t vocab, int64_t rows) {
    const int32_t chunk = kThreads * kVecs * (dtype == KDA_BF16 ? 8 : 4), chunks = (vocab + chunk - 1) / chunk;
    // Long segments leave short lists to join; short ones fill the GPU where there are few rows.
    int32_t each = kMostChunks;
    while (each > 1 && rows * ((chunks + each - 1) / each) < kWaves * device_sm_count()) each /= 2;
    return Layout{(chunks + each - 1) / each, each * chunk};
}

template <typename T>
cudaError_t launch(const BeamSelectArgs &a, const Layout &lay, cudaStream_t stream) {
    return launch_serial(beam_segments_kernel<T, kVecs>, dim3((unsigned)(a.batch * a.beams), (unsigned)lay.segments), kThreads,
                         0, stream, a, lay);
}

}  // namespace

// (the most segments that any call of these sizes has)
size_t beam_select_workspace(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    const int32_t chunk = kThreads * kVecs * 4;
    return (size_t)batch * beams * ((vocab + chunk - 1) / chunk) * segment_words(choices) * 8;
}

cudaError_t launch_beam_select(const BeamSelectArgs &a, cudaStream_t stream) {
    const Layout lay = layout(a.dtype, a.vocab, (int64_t)a.batch * a.beams);
    cudaError_t e = a.dtype == KDA_BF16 ? launch<__nv_bfloat16>(a, lay, stream) : launch<float>(a, lay, stream);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)a.beams * lay.segments;
    if (smem > 16 * 1024) e = allow_smem(beam_join_kernel, kMostLists);
    return e == cudaSuccess ? launch_serial(beam_join_kernel, dim3((unsigned)a.batch), kThreads, smem, stream, a, lay) : e;
}

}  // namespace kda
