// Pages of the key/value cache: copy, fork, release, compact.
//
// Which pages are free is never stored: a page is live when some row of the table names it.
// The two calls that need to know mark the table's entries in a bitmap of P bits, which one
// SM's shared memory holds (128 KB at the limit of 2^20 pages), so one CTA plans the call
//   fork:    k-th fresh page = k-th zero bit
//   compact: L = number of ones; the k-th one at or above L moves to the k-th zero below L
// by prefix sums over the bitmap's words, and leaves a list of (src, dst) moves.  The second
// launch moves the bytes (HBM-bound: each page is read once and written once).  Moved pages and
// their destinations are disjoint sets, so the order of the copies does not matter, and the
// lists depend only on the table, so a call repeats bit for bit.
// Measured: 1,590 of 2,160 pages of 262 KB moved (834 MB read and written) 130 us, 6.4 TB/s, 0.94 of the
// measured copy bandwidth, about 5 us of it the plan; four branches in four layers after a trim of 32
// rows 8.0 us on the device (the two calls from Python: 20 to 24).
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int32_t kRefused = -2;  // in place of a fork's source page
constexpr int64_t kChunk = (int64_t)kCopyThreads * kCopyUnroll * 16;  // 16 KB a work unit

__device__ __forceinline__ bool page_ok(int32_t id, int32_t num_pages) {
    return (uint32_t)id < (uint32_t)num_pages;
}

// ---------------------------------------------------------------------------
// Moving the bytes
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy_pages(const PageMoves &m, int32_t n) {
    const int64_t chunks = (m.page_bytes + kChunk - 1) / kChunk;
    const int64_t units = (int64_t)n * m.num_layers * chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t page, chunk, layer;
        int32_t i;
        if (units <= 0xffffffffLL) {  // 32-bit divisions
            page = (uint32_t)u / (uint32_t)chunks;
            layer = (uint32_t)page / (uint32_t)n;
        } else {
            page = u / chunks;
            layer = page / n;
        }
        chunk = u - page * chunks;
        i = (int32_t)(page - layer * n);
        const int32_t s = m.src[i], d = m.dst[i];
        if (!page_ok(s, m.num_pages) || !page_ok(d, m.num_pages)) continue;
        const int64_t words = m.page_bytes / 16, first = chunk * (kChunk / 16);
        const uint4 *from = static_cast<const uint4 *>(m.pool) + (layer * m.num_pages + s) * words;
        uint4 *to = static_cast<uint4 *>(m.pool) + (layer * m.num_pages + d) * words;
        uint4 x[kCopyUnroll];
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
            const int64_t w = first + k * kCopyThreads + threadIdx.x;
            if (w < words) x[k] = __ldcs(from + w);
        }
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
            const int64_t w = first + k * kCopyThreads + threadIdx.x;
            if (w < words) __stcs(to + w, x[k]);
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PageMoves m) {
    grid_wait();
    copy_pages(m, m.n);
}

// ---------------------------------------------------------------------------
// Planning: bitmap of live pages and prefix sums over it
// ---------------------------------------------------------------------------
// Exclusive prefix sum of x over the CTA; *total gets the sum.  All threads call it.
__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t *warp_sums, int32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    __syncthreads();  // the previous use of warp_sums is over
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int32_t s = warp_sums[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[31];
    return inc - x + (warp ? warp_sums[warp - 1] : 0);
}

// Bits of `word` (number w) that name pages below num_pages.
__device__ __forceinline__ uint32_t valid_bits(int32_t w, int32_t num_pages) {
    const int32_t left = num_pages - w * 32;
    return left >= 32 ? 0xffffffffu : (1u << left) - 1u;
}

// Marks the pages that the rows name; rows whose bit is set in `skip` (may be null) do not count.
__device__ __forceinline__ void mark_live(uint32_t *live, const uint32_t *skip, const int32_t *table,
                                          int32_t rows, int32_t width, int32_t num_pages) {
    constexpr int kAhead = 8;  // entries a thread has in flight
    const int lane = threadIdx.x & 31;
    const auto mark = [&](int32_t id) {
        if (page_ok(id, num_pages)) atomicOr(live + (id >> 5), 1u << (id & 31));
    };
    if (skip == nullptr) {  // the whole table as one array
        const int64_t entries = (int64_t)rows * width;
        for (int64_t e0 = threadIdx.x; e0 < entries; e0 += kAhead * kPlanThreads) {
            int32_t id[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) id[k] = e0 + k * kPlanThreads < entries ? table[e0 + k * kPlanThreads] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) mark(id[k]);
        }
        return;
    }
    for (int32_t r = threadIdx.x >> 5; r < rows; r += kPlanThreads / 32) {  // a warp a row
        if (skip[r >> 5] >> (r & 31) & 1u) continue;
        const int32_t *row = table + (int64_t)r * width;
        for (int32_t c0 = lane; c0 < width; c0 += 32 * kAhead) {
            int32_t id[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) id[k] = c0 + 32 * k < width ? row[c0 + 32 * k] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) mark(id[k]);
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(const PageForkArgs a) {
    extern __shared__ uint32_t smem[];
    __shared__ int32_t warp_sums[32];
    const int32_t P = a.moves.num_pages, R = a.table_rows, M = a.table_width, F = a.moves.n;
    const int32_t words = (P + 31) / 32, row_words = (R + 31) / 32;
    uint32_t *live = smem, *is_child = smem + words;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the copies come up meanwhile
    for (int32_t i = tid; i < words + row_words; i += kPlanThreads) smem[i] = 0;
    grid_wait();
    __syncthreads();
    for (int32_t i = tid; i < F; i += kPlanThreads) {
        const int32_t c = a.child[i];
        if ((uint32_t)c < (uint32_t)R && c != a.parent[i]) atomicOr(is_child + (c >> 5), 1u << (c & 31));
    }
    __syncthreads();
    mark_live(live, is_child, a.page_table, R, M, P);
    __syncthreads();

    // the lowest free pages, as many as there are forks
    const int32_t per = (words + kPlanThreads - 1) / kPlanThreads, w0 = tid * per;
    int32_t mine = 0, total_free;
    for (int32_t w = w0; w < min(w0 + per, words); ++w) mine += __popc(~live[w] & valid_bits(w, P));
    int32_t rank = block_scan(mine, warp_sums, &total_free);
    for (int32_t w = w0; w < min(w0 + per, words) && rank < F; ++w) {
        uint32_t bits = ~live[w] & valid_bits(w, P);
        while (bits != 0 && rank < F) {
            a.free_list[rank++] = w * 32 + __ffs(bits) - 1;
            bits &= bits - 1;
        }
    }
    __syncthreads();  // free_list is read by the whole CTA below

    int32_t used = 0;
    for (int32_t base = 0; base < F; base += kPlanThreads) {
        const int32_t i = base + tid;
        int32_t parent = -1, child = -1, length = 0, last = 0, old = -1;
        bool ok = false, half = false;
        if (i < F) {
            parent = a.parent[i];
            child = a.child[i];
            ok = (uint32_t)parent < (uint32_t)R && (uint32_t)child < (uint32_t)R && parent != child;
            if (ok) {
                length = a.kv_len[parent];
                ok = length >= 0 && length <= M * a.page_size;
            }
            if (ok && length % a.page_size != 0) {
                last = length / a.page_size;  // < M: length <= M page_size and not a multiple
                old = a.page_table[(int64_t)parent * M + last];
                half = page_ok(old, P);
            }
        }
        int32_t wanted;
        const int32_t k = used + block_scan(half ? 1 : 0, warp_sums, &wanted);
        used += wanted;
        if (i < F) {
            if (half && k >= total_free) ok = half = false;  // no page left for it
            const int32_t fresh = half ? a.free_list[k] : -1;
            a.src[i] = !ok ? kRefused : half ? old : -1;
            a.dst[i] = fresh;
            if (!ok) record_status(a.status, KDA_ERR_DEVICE_CHECK, (uint32_t)i);
            if ((uint32_t)child < (uint32_t)R && child != parent) a.kv_len[child] = ok ? length : 0;
        }
        __syncthreads();
        // the rows of this batch of forks, a warp a row
        for (int32_t f = base + (tid >> 5); f < min(base + kPlanThreads, F); f += kPlanThreads / 32) {
            const int32_t p = a.parent[f], c = a.child[f];
            if ((uint32_t)c >= (uint32_t)R || c == p) continue;
            int32_t *to = a.page_table + (int64_t)c * M;
            const bool given = a.src[f] != kRefused;
            const int32_t fresh = a.dst[f], length = a.kv_len[c];
            const int32_t at = fresh >= 0 ? length / a.page_size : -1;
            // what the parent has mapped past its tokens stays its own: both rows would append there
            const int32_t shared = given ? length / a.page_size + (length % a.page_size != 0) : 0;
            for (int32_t j = tid & 31; j < M; j += 32)
                to[j] = j >= shared ? -1 : j == at ? fresh : a.page_table[(int64_t)p * M + j];
        }
        __syncthreads();
    }
}

// The plan of a compaction: moves in (src, dst), the new name of every page that moves in remap.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(const PageCompactArgs a) {
    extern __shared__ uint32_t smem[];
    __shared__ int32_t warp_sums[32];
    const int32_t P = a.moves.num_pages, words = (P + 31) / 32;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the moves come up meanwhile
    for (int32_t i = tid; i < words; i += kPlanThreads) smem[i] = 0;
    grid_wait();
    __syncthreads();
    mark_live(smem, nullptr, a.table_in, a.table_rows, a.table_width, P);
    __syncthreads();
    const int32_t per = (words + kPlanThreads - 1) / kPlanThreads;
    const int32_t w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int32_t mine = 0, live;
    for (int32_t w = w0; w < w1; ++w) mine += __popc(smem[w]);
    const int32_t before = block_scan(mine, warp_sums, &live);
    // ones below L, and the ranks of this thread's holes and movers
    int32_t below = 0;
    for (int32_t w = w0; w < w1; ++w) below += __popc(smem[w] & valid_bits(w, live < w * 32 ? w * 32 : live));
    int32_t all_below;
    const int32_t below_before = block_scan(below, warp_sums, &all_below);
    int32_t hole = min(w0 * 32, live) - below_before;  // zeros below L before word w0
    int32_t mover = before - below_before;             // ones at or above L before word w0
    for (int32_t w = w0; w < w1; ++w) {
        const uint32_t under = valid_bits(w, live < w * 32 ? w * 32 : live);
        for (uint32_t z = ~smem[w] & under; z != 0; z &= z - 1) a.dst[hole++] = w * 32 + __ffs(z) - 1;
        for (uint32_t o = smem[w] & ~under; o != 0; o &= o - 1) a.src[mover++] = w * 32 + __ffs(o) - 1;
    }
    __syncthreads();
    const int32_t moves = live - all_below;
    for (int32_t i = tid; i < moves; i += kPlanThreads) a.remap[a.src[i]] = a.dst[i];
    if (tid == 0) {
        *a.count = moves;
        *a.num_live = live;
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_compact_move_kernel(const PageCompactArgs a) {
    grid_wait();
    const int32_t live = *a.num_live, P = a.moves.num_pages;
    const int64_t entries = (int64_t)a.table_rows * a.table_width;
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < entries;
         i += (int64_t)gridDim.x * kCopyThreads) {
        const int32_t id = a.table_in[i];
        a.table_out[i] = page_ok(id, P) && id >= live ? a.remap[id] : id;
    }
    copy_pages(a.moves, *a.count);
}

constexpr int kReleaseThreads = 128;

__global__ void __launch_bounds__(kReleaseThreads) pages_release_kernel(const PageReleaseArgs a) {
    grid_wait();
    const int32_t r = a.rows[blockIdx.x];
    if ((uint32_t)r >= (uint32_t)a.table_rows) {
        if (threadIdx.x == 0) record_status(a.status, KDA_ERR_DEVICE_CHECK, blockIdx.x);
        return;
    }
    int32_t *row = a.page_table + (int64_t)r * a.table_width;
    int64_t from = 0, to = a.table_width;  // entries [from, to) go
    if (a.window > 0) {
        // a token to come (index >= kv_len) sees j > kv_len - window, and j < sinks
        from = ((int64_t)a.sinks + a.page_size - 1) / a.page_size;
        to = min(to, max((int64_t)0, (int64_t)a.kv_len[r] - a.window + 1) / a.page_size);
    } else if (threadIdx.x == 0) {
        a.kv_len[r] = 0;
    }
    for (int64_t j = from + threadIdx.x; j < to; j += kReleaseThreads) row[j] = -1;
}

// Shared memory of a plan: a bit a page, and for a fork a bit a row.  Above 32 KB (with the static
// arrays still well inside the default 48) the kernel gets the most that the calls accept, 160 KB.
constexpr size_t kPlanSmem = ((1 << 20) + (1 << 18)) / 8;
template <typename Args>
cudaError_t launch_plan(void (*kernel)(Args), size_t smem, cudaStream_t stream, const Args &a) {
    if (smem > 32 * 1024) {
        const cudaError_t e = allow_smem(kernel, kPlanSmem);
        if (e != cudaSuccess) return e;
    }
    return launch_serial(kernel, dim3(1), kPlanThreads, smem, stream, a);
}

unsigned copy_grid(int64_t units) {
    const int64_t most = (int64_t)device_sm_count() * 64;
    return (unsigned)(units < 1 ? 1 : units < most ? units : most);
}
int64_t copy_units(const PageMoves &m, int64_t n) {
    return n * m.num_layers * ((m.page_bytes + kChunk - 1) / kChunk);
}
}  // namespace

cudaError_t launch_pages_copy(const PageMoves &m, cudaStream_t stream) {
    if (m.n == 0) return cudaSuccess;
    return launch_serial(pages_copy_kernel, dim3(copy_grid(copy_units(m, m.n))), kCopyThreads, 0, stream, m);
}

cudaError_t launch_pages_fork(const PageForkArgs &a, cudaStream_t stream) {
    if (a.moves.n == 0) return cudaSuccess;
    const size_t smem = 4 * (((size_t)a.moves.num_pages + 31) / 32 + ((size_t)a.table_rows + 31) / 32);
    const cudaError_t e = launch_plan(pages_fork_plan_kernel, smem, stream, a);
    return e == cudaSuccess ? launch_pages_copy(a.moves, stream) : e;
}

cudaError_t launch_pages_release(const PageReleaseArgs &a, cudaStream_t stream) {
    if (a.n == 0) return cudaSuccess;
    return launch_serial(pages_release_kernel, dim3((unsigned)a.n), kReleaseThreads, 0, stream, a);
}

cudaError_t launch_pages_compact(const PageCompactArgs &a, cudaStream_t stream) {
    const size_t smem = 4 * (((size_t)a.moves.num_pages + 31) / 32);
    const cudaError_t e = launch_plan(pages_compact_plan_kernel, smem, stream, a);
    if (e != cudaSuccess) return e;
    // at most min(L, P - L) <= P / 2 pages move
    const unsigned grid = copy_grid(copy_units(a.moves, (a.moves.num_pages + 1) / 2));
    return launch_serial(pages_compact_move_kernel, dim3(grid), kCopyThreads, 0, stream, a);
}

}  // namespace kda
