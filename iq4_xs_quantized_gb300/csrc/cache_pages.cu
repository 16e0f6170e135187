// cache_pages.cu -- the cache's page operations: reserve, commit (compact and
// free), fork, release and page copies.
//
// A page is free when its reference count is zero.  Allocation is a rank
// match: the r-th free page (rising index) goes to the r-th page that the
// requests, in order, ask for; one CTA counts the free pages of a chunk by a
// block scan and looks each rank up in the running sum of the requests, so
// the result does not depend on timing.  Counts fall and rise by integer
// atomics, whose order does not matter.  Moving and copying K and V is bound
// by HBM (each byte read once and written once), small calls by the loads that
// wait for one another: row, length, page, data.
//
// Measured: fork of 4 parents of 700 tokens by 8, 64 layers of 4 heads of 256,
// 482 MB in 80.5 us, 5.99 TB/s (88 % of a copy's rate); commit of 7 of 16
// tokens of 32 sequences in the same cache, 42 MB in 17.5-19.4 us (2.2-2.4
// TB/s), of 4 tokens of one sequence in 8 layers 5.6 us; fork of one by two
// there 10.7 us.  Long ones stay far off: every thread of a commit walks the
// whole path (a chain of 512 tokens 69 us, of 8,000 1.05 ms), and a fork's books
// are one CTA's (one child of 100,000 tokens in pages of 16: 42 us).
#include "cache.cuh"

namespace iq4xs {
namespace {

constexpr int kBookThreads = 1024;
constexpr int kPagesPerThread = 16;

// Exclusive sum of v over the block and the block's total.
__device__ int block_scan(int v, int* total) {
    __shared__ int warp_sum[32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) warp_sum[w] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
        const int t = warp_sum[i];
        before += i < w ? t : 0;
        all += t;
    }
    *total = all;
    return before + x - v;
}

// Free pages of the thread's kPagesPerThread pages from `first` on, as bits.
__device__ uint32_t free_bits(const Bc& bc, const int32_t* refs, int64_t first, int pages) {
    uint32_t bits = 0;
    if (first + kPagesPerThread <= pages) {
        int4 r[kPagesPerThread / 4];
#pragma unroll
        for (int i = 0; i < kPagesPerThread / 4; ++i)
            r[i] = bc_global(bc, refs + first + 4 * i, 16, refs, 4 * (int64_t)pages, kBcPagesRefs)
                       ? *reinterpret_cast<const int4*>(refs + first + 4 * i)
                       : make_int4(1, 1, 1, 1);
#pragma unroll
        for (int i = 0; i < kPagesPerThread / 4; ++i)
            bits |= ((r[i].x == 0) | (r[i].y == 0) << 1 | (r[i].z == 0) << 2 | (r[i].w == 0) << 3) << (4 * i);
    } else {
        for (int i = 0; i < kPagesPerThread && first + i < pages; ++i)
            if (bc_global(bc, refs + first + i, 4, refs, 4 * (int64_t)pages, kBcPagesRefs))
                bits |= (uint32_t)(refs[first + i] == 0) << i;
    }
    return bits;
}

// Free pages, counted up to `wanted` (the scan stops there).
__device__ int count_free(const Bc& bc, const int32_t* refs, int pages, int wanted) {
    int found = 0;
    for (int64_t c0 = 0; c0 < pages && found < wanted; c0 += kBookThreads * kPagesPerThread) {
        int total;
        block_scan(__popc(free_bits(bc, refs, c0 + (int64_t)threadIdx.x * kPagesPerThread, pages)), &total);
        found += total;
    }
    return found;
}

// give(rank, page) for the free pages of rank 0..fit-1 in rising order, each
// by one thread, where fit = wanted if that many are free, else what
// fit_of(free pages) says.  Returns fit.
template <class Fit, class Give>
__device__ int hand_out(const Bc& bc, const int32_t* refs, int pages, int wanted, Fit fit_of, Give give) {
    // Mostly the first pages looked at hold enough: then they need no second look.
    uint32_t bits = free_bits(bc, refs, (int64_t)threadIdx.x * kPagesPerThread, pages);
    int total;
    int rank = block_scan(__popc(bits), &total);
    const auto give_all = [&](int64_t first, int fit) {
        for (; bits && rank < fit; bits &= bits - 1, ++rank) give(rank, (int)(first + __ffs(bits) - 1));
    };
    int fit = wanted;
    if (total < wanted) {
        const int nfree = count_free(bc, refs, pages, wanted);
        if (nfree < wanted) fit = fit_of(nfree);
        __syncthreads();  // every count is done before a page changes hands
    }
    give_all((int64_t)threadIdx.x * kPagesPerThread, fit);
    int rank0 = total;
    for (int64_t c0 = kBookThreads * kPagesPerThread; c0 < pages && rank0 < fit; c0 += kBookThreads * kPagesPerThread) {
        const int64_t first = c0 + (int64_t)threadIdx.x * kPagesPerThread;
        bits = free_bits(bc, refs, first, pages);
        rank = rank0 + block_scan(__popc(bits), &total);
        give_all(first, fit);
        rank0 += total;
    }
    return fit;
}

// First i with upto[i] > rank (upto does not fall; upto[n - 1] > rank).
__device__ int find_taker(const int32_t* upto, int n, int rank) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > rank) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_for(int64_t tokens, int shift) {
    return (int)((tokens + (int64_t(1) << shift) - 1) >> shift);
}

// Pages that sequence s lacks for its new tokens; -1: more than its table
// holds, or values out of range (recorded).
__device__ int pages_lacking(const BatchView& b, int s, int shift, int* held_out, int* err) {
    int first;
    const int n = batch_rows(b, s, INT32_MAX, &first, err);
    const int len = batch_len(b, s, err), held = b.held[s];
    *held_out = held;
    if (held < 0 || held > b.table_width) data_error(err, kDataHeld);
    if (len < 0 || held < 0 || held > b.table_width) return -1;
    const int want = pages_for((int64_t)len + n, shift);
    return want > b.table_width ? -1 : max(0, want - held);
}

__global__ void __launch_bounds__(kBookThreads)
    reserve_kernel(const BatchView b, int shift, int32_t* refs, int pages, int32_t* status, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    // The running sum of the requests: in shared memory, or where there are
    // more sequences than it holds in status, until the end.
    __shared__ int32_t upto_s[kBookThreads];
    int32_t* const upto = b.sequences <= kBookThreads ? upto_s : status;
    int wanted = 0;
    for (int s0 = 0; s0 < b.sequences; s0 += kBookThreads) {
        const int s = s0 + threadIdx.x;
        int held;
        const int lack = s < b.sequences ? max(0, pages_lacking(b, s, shift, &held, err)) : 0;
        int total;
        const int before = block_scan(lack, &total);
        // (sums past the number of pages are all alike: nothing fits there)
        if (s < b.sequences) upto[s] = (int)min((int64_t)INT32_MAX, (int64_t)wanted + before + lack);
        wanted = (int)min((int64_t)INT32_MAX, (int64_t)wanted + total);
    }
    __syncthreads();
    int fit = wanted;  // pages handed out: those of the sequences before the first that does not fit
    if (wanted > 0) {
        fit = hand_out(
            bc, refs, pages, wanted,
            [&](int nfree) {
                const int i = find_taker(upto, b.sequences, nfree);
                return i > 0 ? upto[i - 1] : 0;
            },
            [&](int rank, int page) {
                const int s = find_taker(upto, b.sequences, rank);
                const int at = b.held[s] + rank - (s > 0 ? upto[s - 1] : 0);
                int32_t* to = b.page_table + s * b.table_stride + at;
                if (bc_range(bc, at, 1, b.table_width, kBcPagesTable)) *to = page;
                refs[page] = 1;
            });
        __syncthreads();
    }
    for (int s0 = 0; s0 < b.sequences; s0 += kBookThreads) {
        const int s = s0 + threadIdx.x;
        if (s < b.sequences) {
            int held;
            const int lack = pages_lacking(b, s, shift, &held, err);
            const bool ok = lack == 0 || (lack > 0 && upto[s] <= fit);
            if (ok && lack > 0) b.held[s] = held + lack;
            status[s] = ok ? 0 : 1;
        }
    }
}

// One reference less to `page`.  A count that is zero already stays zero, and
// is reported: the page would otherwise never be free again.
__device__ __forceinline__ void drop_page(const Bc& bc, int32_t* refs, int page, int pages, int* err) {
    if (page < 0 || page >= pages) {
        data_error(err, kDataPage);
    } else if (bc_global(bc, refs + page, 4, refs, 4 * (int64_t)pages, kBcPagesRefs)) {
        if (atomicSub(refs + page, 1) <= 0) {
            atomicAdd(refs + page, 1);
            data_error(err, kDataRefs);
        }
    }
}

// ------------------------------------------------------------------ commit
// One thread per 16-byte column of a head's row: it walks the accepted path
// of its sequence in order, up to kMoveBatch loads in flight before their
// stores.  Paths rise strictly, so path[i] >= i and a store to place i never
// overtakes a load that is still to come (those read places >= i + 1).
constexpr int kMoveThreads = 512;
constexpr int kMoveBatch = 8;
constexpr int kMoveRows = 64;  // rows of the path looked up at a time

__device__ bool path_ok(const int32_t* path, int n, int width, int tokens, int len) {
    if (n < 0 || n > width || len < 0 || len > INT32_MAX - tokens) return false;
    int last = -1;
    for (int i = 0; i < n; ++i) {
        const int p = path[i];
        if (p <= last || p >= tokens) return false;
        last = p;
    }
    return true;
}

// A cluster per sequence shares its columns; its first CTA then keeps the
// books, once every CTA is done with what it rewrites (held, and the length
// when new_lens is lens): one launch where two would follow each other.
__global__ void __launch_bounds__(kMoveThreads)
    commit_kernel(const CacheView c, const BatchView b, int32_t* refs, const int32_t* paths, int width,
                  const int32_t* accepted, int32_t* new_lens, int* err) {
    __shared__ int64_t from_s[kMoveRows], to_s[kMoveRows];
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int s = blockIdx.y;
    int first;
    const int tokens = batch_rows(b, s, INT32_MAX, &first, err);
    const int len = b.lens[s], n = accepted[s], held = b.held[s];
    const int32_t* path = paths + (int64_t)s * width;
    // (rows that stay where they are look no page up: their end is compared with the pages held)
    const bool held_ok = held >= 0 && held <= b.table_width && (int64_t)len + n <= (int64_t)held << c.page_shift;
    const bool ok = path_ok(path, n, width, tokens, len) && held_ok;
    // 16-byte columns of a row, and segments (layer, K or V, head), fewer than
    // 2^28: 32-bit divisions cost a tenth of 64-bit ones.
    const int cols = c.head_dim / 8, stride = gridDim.x * kMoveThreads / cols;
    const uint32_t segs = ok ? (uint32_t)(c.layers * 2 * c.heads) : 0u;
    for (int c0 = 0; ok && c0 < n; c0 += kMoveRows) {
        // where the next rows of the path lie in a (layer, head), -1: stays or cannot move
        __syncthreads();
        if (threadIdx.x < kMoveRows) {
            const int i = c0 + threadIdx.x;
            int64_t f = -1, t = -1;
            if (i < n && path[i] != i) {
                const int src = len + path[i], dst = len + i;
                const int ps = page_of(c, b, s, src, err), pd = page_of(c, b, s, dst, err);
                if (ps >= 0 && pd >= 0) {
                    f = ps * c.page_stride + (src & (c.page_size - 1)) * c.slot_stride;
                    t = pd * c.page_stride + (dst & (c.page_size - 1)) * c.slot_stride;
                }
            }
            from_s[threadIdx.x] = f;
            to_s[threadIdx.x] = t;
        }
        __syncthreads();
        const int rows = min(kMoveRows, n - c0);
        for (uint32_t seg = (blockIdx.x * kMoveThreads + threadIdx.x) / cols; seg < segs; seg += stride) {
            const uint32_t side = seg / c.heads, head = seg - side * c.heads;
            uint16_t* base = side % 2 ? c.v : c.k;
            uint16_t* column = base + (side / 2) * c.layer_stride + head * c.head_stride + threadIdx.x % cols * 8;
            for (int i0 = 0; i0 < rows; i0 += kMoveBatch) {
                uint4 val[kMoveBatch];
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k)
                    if (i0 + k < rows && from_s[i0 + k] >= 0 &&
                        bc_global(bc, column + from_s[i0 + k], 16, base, c.extent, kBcPagesKv))
                        val[k] = *reinterpret_cast<const uint4*>(column + from_s[i0 + k]);
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k)
                    if (i0 + k < rows && to_s[i0 + k] >= 0 &&
                        bc_global(bc, column + to_s[i0 + k], 16, base, c.extent, kBcPagesKv))
                        *reinterpret_cast<uint4*>(column + to_s[i0 + k]) = val[k];
            }
        }
    }
    cluster_arrive_release();
    cluster_wait();
    if (blockIdx.x != 0) return;
    if (!ok) {
        if (threadIdx.x == 0) {
            data_error(err, len < 0 ? kDataLens : held_ok ? kDataPath : kDataHeld);
            new_lens[s] = len;
        }
        return;
    }
    const int keep = min(held, pages_for((int64_t)len + n, c.page_shift));
    for (int j = keep + threadIdx.x; j < held; j += kMoveThreads)
        drop_page(bc, refs, b.page_table[s * b.table_stride + j], c.pages, err);
    if (threadIdx.x == 0) {
        b.held[s] = keep;
        new_lens[s] = len + n;
    }
}

// -------------------------------------------------------------------- fork
// A child's full pages to share and pages to take, 0 or 1; 2 where its indices
// or counts are out of order, else 0.
__device__ int fork_state(const BatchView& b, int parent, int child, int shift, int* full, int* take) {
    *full = *take = 0;
    if (parent < 0 || parent >= b.sequences || child < 0 || child >= b.sequences || parent == child) return 2;
    const int len = b.lens[parent];
    if (len < 0 || b.held[child] != 0) return 2;
    const int need = pages_for(len, shift);
    if (need > b.held[parent] || b.held[parent] > b.table_width) return 2;
    *full = len >> shift;
    *take = need - *full;
    return 0;
}

__global__ void __launch_bounds__(kBookThreads)
    fork_book_kernel(const BatchView b, int shift, int32_t* refs, int pages, const int32_t* parents,
                     const int32_t* children, int count, int32_t* status, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    // the running sum of the requests, as in reserve_kernel
    __shared__ int32_t upto_s[kBookThreads];
    int32_t* const upto_all = count <= kBookThreads ? upto_s : status;
    int wanted = 0;
    for (int i0 = 0; i0 < count; i0 += kBookThreads) {
        const int i = i0 + threadIdx.x;
        int full, take = 0;
        if (i < count) fork_state(b, parents[i], children[i], shift, &full, &take);
        int total;
        const int before = block_scan(take, &total);
        if (i < count) upto_all[i] = wanted + before + take;
        wanted += total;
    }
    __syncthreads();
    int fit = wanted;
    if (wanted > 0) {
        fit = hand_out(
            bc, refs, pages, wanted, [](int nfree) { return nfree; },
            [&](int rank, int page) {
                const int i = find_taker(upto_all, count, rank);
                int full, take;
                fork_state(b, parents[i], children[i], shift, &full, &take);
                if (bc_range(bc, full, 1, b.table_width, kBcPagesTable))
                    b.page_table[children[i] * b.table_stride + full] = page;
                refs[page] = 1;
            });
        __syncthreads();
    }
    // A warp per child: the shared pages' entries and references.
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < count; i0 += kBookThreads / 32) {
        const int i = i0 + (threadIdx.x >> 5);
        int full = 0, take = 0, bad = 0, upto = 0;
        if (i < count) {
            upto = upto_all[i];
            bad = fork_state(b, parents[i], children[i], shift, &full, &take);
            if (!bad && take && upto > fit) bad = 1;
            if (!bad) {
                const int32_t* from = b.page_table + parents[i] * b.table_stride;
                int32_t* to = b.page_table + children[i] * b.table_stride;
                for (int j = lane; j < full; j += 32) {
                    const int page = from[j];
                    to[j] = page;
                    if (page < 0 || page >= pages) data_error(err, kDataPage);
                    else if (bc_global(bc, refs + page, 4, refs, 4 * (int64_t)pages, kBcPagesRefs))
                        atomicAdd(refs + page, 1);
                }
            }
        }
        __syncthreads();
        if (i < count && lane == 0) {
            if (bad == 2) data_error(err, kDataRow);
            if (!bad) {
                b.held[children[i]] = full + take;
                b.lens[children[i]] = b.lens[parents[i]];
            }
            status[i] = bad;
        }
    }
}

// ------------------------------------------------------------------- copies
constexpr int kCopyThreads = 128;
constexpr int kCopyBatch = 4;

// `slots` slots of one (layer, K or V, head) from page `src` to page `dst`.
__device__ void copy_slots(const Bc& bc, const CacheView& c, uint32_t seg, int src, int dst, int slots) {
    const int cols = c.head_dim / 8;
    const uint32_t side = seg / c.heads, head = seg - side * c.heads;
    uint16_t* base = side % 2 ? c.v : c.k;
    uint16_t* rows = base + (side / 2) * c.layer_stride + head * c.head_stride;
    const uint16_t* from = rows + src * c.page_stride;
    uint16_t* to = rows + dst * c.page_stride;
    const int units = slots * cols;
    for (int u0 = threadIdx.x; u0 < units; u0 += kCopyThreads * kCopyBatch) {
        uint4 val[kCopyBatch];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k) {
            const int u = u0 + k * kCopyThreads;
            const uint16_t* f = from + (u / cols) * c.slot_stride + (u % cols) * 8;
            if (u < units && bc_global(bc, f, 16, base, c.extent, kBcPagesKv))
                val[k] = __ldcs(reinterpret_cast<const uint4*>(f));
        }
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k) {
            const int u = u0 + k * kCopyThreads;
            uint16_t* t = to + (u / cols) * c.slot_stride + (u % cols) * 8;
            if (u < units && bc_global(bc, t, 16, base, c.extent, kBcPagesKv)) *reinterpret_cast<uint4*>(t) = val[k];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(const CacheView c, const BatchView b, const int32_t* parents,
                     const int32_t* children, const int32_t* status, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int i = blockIdx.y;
    if (status[i] != 0) return;
    const int parent = parents[i], child = children[i];
    const int len = b.lens[parent], tail = len & (c.page_size - 1);
    if (tail == 0) return;
    const int src = page_of(c, b, parent, len, err), dst = page_of(c, b, child, len, err);
    if (src >= 0 && dst >= 0) copy_slots(bc, c, blockIdx.x, src, dst, tail);
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const CacheView c, const int32_t* src, const int32_t* dst, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int a = src[blockIdx.y], z = dst[blockIdx.y];
    if (a < 0 || a >= c.pages || z < 0 || z >= c.pages) {
        data_error(err, kDataPage);
        return;
    }
    if (a != z) copy_slots(bc, c, blockIdx.x, a, z, c.page_size);
}

constexpr int kReleaseThreads = 256;

__global__ void __launch_bounds__(kReleaseThreads)
    release_kernel(const BatchView b, int32_t* refs, int pages, const int32_t* rows, int* err) {
    __shared__ int held_s;
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int s = rows[blockIdx.x];
    if (s < 0 || s >= b.sequences) {
        data_error(err, kDataRow);
        return;
    }
    // The count is taken away in one step, so that a sequence named twice
    // drops its references once.
    if (threadIdx.x == 0) {
        held_s = atomicExch(b.held + s, 0);
        b.lens[s] = 0;
    }
    __syncthreads();
    int held = held_s;
    if (held < 0 || held > b.table_width) {
        data_error(err, kDataHeld);
        held = 0;
    }
    for (int j = threadIdx.x; j < held; j += kReleaseThreads)
        drop_page(bc, refs, b.page_table[s * b.table_stride + j], pages, err);
}

}  // namespace

cudaError_t launch_cache_reserve(const BatchView& b, int page_size, int32_t* refs, int pages, int32_t* status, int* err,
                                 cudaStream_t stream) {
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    return launch_chained(reserve_kernel, dim3(1), dim3(kBookThreads), 0, stream, 1, b, shift, refs, pages, status, err);
}

cudaError_t launch_cache_commit(const CacheView& c, const BatchView& b, int32_t* refs, const int32_t* paths,
                                int path_width, const int32_t* accepted, int32_t* new_lens, int* err,
                                cudaStream_t stream) {
    // One CTA a sequence up to the portable eight: as many as its columns fill.
    const int64_t units = (int64_t)c.layers * 2 * c.heads * (c.head_dim / 8);
    const int64_t full = (units + kMoveThreads - 1) / kMoveThreads;
    const unsigned ctas = full >= 8 ? 8 : full >= 4 ? 4 : full >= 2 ? 2 : 1;
    return launch_chained(commit_kernel, dim3(ctas, (unsigned)b.sequences), dim3(kMoveThreads), 0, stream, (int)ctas, c,
                          b, refs, paths, path_width, accepted, new_lens, err);
}

cudaError_t launch_cache_fork(const CacheView& c, const BatchView& b, int32_t* refs, const int32_t* parents,
                              const int32_t* children, int count, int32_t* status, int* err, cudaStream_t stream) {
    const cudaError_t e = launch_chained(fork_book_kernel, dim3(1), dim3(kBookThreads), 0, stream, 1, b, c.page_shift,
                                         refs, c.pages, parents, children, count, status, err);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(c.layers * 2 * c.heads), (unsigned)count);
    return launch_chained(fork_copy_kernel, grid, dim3(kCopyThreads), 0, stream, 1, c, b, parents, children,
                          (const int32_t*)status, err);
}

cudaError_t launch_cache_copy_pages(const CacheView& c, const int32_t* src, const int32_t* dst, int count, int* err,
                                    cudaStream_t stream) {
    const dim3 grid((unsigned)(c.layers * 2 * c.heads), (unsigned)count);
    return launch_chained(copy_pages_kernel, grid, dim3(kCopyThreads), 0, stream, 1, c, src, dst, err);
}

cudaError_t launch_cache_release(const BatchView& b, int32_t* refs, int pages, const int32_t* rows, int count,
                                 int* err, cudaStream_t stream) {
    return launch_chained(release_kernel, dim3((unsigned)count), dim3(kReleaseThreads), 0, stream, 1, b, refs, pages, rows,
                          err);
}

}  // namespace iq4xs
