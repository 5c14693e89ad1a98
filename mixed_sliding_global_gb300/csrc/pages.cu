// pages.cu -- pages of a pool: sharing them between sequences, giving private ones to the
// positions that are about to be written, taking them back, and moving the used ones together.
//
// The block table [batch][max_pages] (a negative entry: no page) and a reference count per page
// are the whole state: a page is free while its count is 0. New pages are the lowest free ones in
// the order of (sequence, position), so results do not depend on scheduling; there is no list of
// free pages that could disagree with the counts.
//
// The bookkeeping is integers of a few dozen to some thousand entries: latency bound. Reserve and
// compact plan in one CTA (its phases are block barriers instead of launches) and leave a list of
// copies in the workspace; a second launch moves the rows of every pool, bandwidth bound, with
// 16-byte accesses, kCopyBytes of them in flight per CTA.
#include <climits>

#include "common.cuh"
#include "tree.h"

namespace gemma {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyBytes = kCopyThreads * kCopyUnroll * 16;  // 32 KB: one unit of the copy launch
constexpr int kPoolsPerLaunch = 128;                         // pools in a launch's arguments
constexpr int kKeeper = 1 << 30;  // reserve's second mark (page numbers are at most kMaxPages)
static_assert(kMaxPages <= kKeeper / 2, "marks of pages");

// Workspace of reserve and compact.
struct Workspace {
    int* n_copies;  // [1]
    int4* copies;   // [n_pages] (source page, destination page, rows, -)
    int* list;      // [n_pages] reserve: free pages; compact: new place of page i
    int* first;     // [n_pages] reserve: the first writer of a shared page
    int* spare;     // [n_pages] compact: source pages
};
__host__ __device__ inline Workspace carve(void* base, int n_pages) {
    const size_t n = ((size_t)n_pages + 3) / 4 * 4;
    Workspace w;
    w.n_copies = static_cast<int*>(base);
    w.copies = reinterpret_cast<int4*>(static_cast<char*>(base) + 256);
    w.list = reinterpret_cast<int*>(w.copies + n);
    w.first = w.list + n;
    w.spare = w.first + n;
    return w;
}

// Exclusive prefix sum of v over the CTA's threads; *total gets the whole sum.
__device__ int block_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // an earlier scan's readers of s_warp are done
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int x = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        s_warp[lane] = x;
    }
    __syncthreads();
    *total = s_warp[kPlanThreads / 32 - 1];
    return incl - v + (warp ? s_warp[warp - 1] : 0);
}

}  // namespace

// ---------------------------------------------------------------------------------------------
// free: entries of pages that hold no position in [keep_from, keep_to) give their page back
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    pages_free_kernel(const PageTable t, const int32_t* __restrict__ keep_from,
                      const int32_t* __restrict__ keep_to, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    const int total = t.batch * t.max_pages;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int b = (int)(i / t.max_pages), blk = (int)(i - (long long)b * t.max_pages);
        // the page's positions within the bounds
        long long begin = (long long)blk * t.page_size, end = begin + t.page_size;
        if (keep_from) begin = max(begin, (long long)__ldg(keep_from + b));
        if (keep_to) end = min(end, (long long)__ldg(keep_to + b));
        if (begin < end) continue;
        const int page = t.table[i];
        if (page < 0) continue;
        if (page >= t.n_pages) {
            report(err, GEMMA_DEVERR_PAGE);
            continue;
        }
        t.table[i] = -1;
        if (atomicSub(t.refs + page, 1) <= 0) {  // nobody held it: the count stays
            atomicAdd(t.refs + page, 1);
            report(err, GEMMA_DEVERR_PAGE);
        }
    }
}

cudaError_t launch_pages_free(const PageTable& t, const int32_t* keep_from, const int32_t* keep_to,
                              uint32_t* err, int n_sm, cudaStream_t st) {
    const long long total = (long long)t.batch * t.max_pages;
    long long blocks = (total + 255) / 256;
    if (blocks > 8ll * n_sm) blocks = 8ll * n_sm;
    return launch_pdl(pages_free_kernel, dim3((unsigned)blocks), dim3(256), 0, st, t, keep_from,
                      keep_to, err);
}

// ---------------------------------------------------------------------------------------------
// fork: a sequence without pages gets the pages of another one's rows
// ---------------------------------------------------------------------------------------------
// One CTA per fork. It refuses its fork, before it writes anything, where the destination is a
// source of the call or an earlier fork's destination, or holds a page: all CTAs judge by what the
// call was given (sources and destinations are never the same row), so their order does not matter.
__global__ void __launch_bounds__(256)
    pages_fork_kernel(const PageTable t, int32_t* seq_lens, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int n, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    const int f = blockIdx.x;
    const int s = __ldg(src + f), d = __ldg(dst + f);
    bool bad = s < 0 || s >= t.batch || d < 0 || d >= t.batch;
    for (int i = threadIdx.x; i < n; i += 256)
        bad |= __ldg(src + i) == d || (i < f && __ldg(dst + i) == d);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report(err, GEMMA_DEVERR_FORK);
        return;
    }
    const int len = seq_lens[s];
    int32_t* to = t.table + (size_t)d * t.max_pages;
    const int32_t* from = t.table + (size_t)s * t.max_pages;
    bool held = false;
    for (int i = threadIdx.x; i < t.max_pages; i += 256) held |= to[i] >= 0;
    const bool bad_len = len < 0 || len > (long long)t.max_pages * t.page_size;
    if (__syncthreads_or(held) || bad_len) {
        if (threadIdx.x == 0) report(err, bad_len ? GEMMA_DEVERR_SEQ_LEN : GEMMA_DEVERR_FORK);
        return;
    }
    const int blocks = (int)(((long long)len + t.page_size - 1) / t.page_size);
    for (int i = threadIdx.x; i < t.max_pages; i += 256) {
        int page = i < blocks ? from[i] : -1;
        if (page >= t.n_pages) {
            report(err, GEMMA_DEVERR_PAGE);
            page = -1;
        }
        if (page >= 0) atomicAdd(t.refs + page, 1);
        to[i] = page < 0 ? -1 : page;
    }
    if (threadIdx.x == 0) seq_lens[d] = len;
}

cudaError_t launch_pages_fork(const PageTable& t, int32_t* seq_lens, const int32_t* src,
                              const int32_t* dst, int n, uint32_t* err, cudaStream_t st) {
    return launch_pdl(pages_fork_kernel, dim3((unsigned)n), dim3(256), 0, st, t, seq_lens, src, dst,
                      n, err);
}

// ---------------------------------------------------------------------------------------------
// copies of pages
// ---------------------------------------------------------------------------------------------
struct CopyPools {
    uint8_t* pool[kPoolsPerLaunch];
    int32_t n_kv[kPoolsPerLaunch];
    int32_t row_bytes[kPoolsPerLaunch];
    int32_t unit0[kPoolsPerLaunch + 1];  // units of a copy before this pool
    int n;
};

// Bytes [0, bytes) of src to dst, both 16-byte aligned, bytes even; the whole CTA.
__device__ __forceinline__ void copy_span(uint8_t* dst, const uint8_t* src, int bytes) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    const int n = bytes / 16;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
        if (threadIdx.x + j * kCopyThreads < n) v[j] = __ldcs(s + threadIdx.x + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
        if (threadIdx.x + j * kCopyThreads < n) __stcs(d + threadIdx.x + j * kCopyThreads, v[j]);
    const int tail = (bytes - 16 * n) / 2;  // rows of less than 16 bytes
    if ((int)threadIdx.x < tail)
        reinterpret_cast<uint16_t*>(dst + 16 * n)[threadIdx.x] =
            reinterpret_cast<const uint16_t*>(src + 16 * n)[threadIdx.x];
}

// Copies of whole pages (compact: one unit is kCopyBytes of a page) or of the first rows of every
// head (reserve: of a head's rows). Compact also gives the table the pages' new places; it looks at every
// entry, moves or not, since an entry of no page in use is reported.
template <bool WHOLE>
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const __grid_constant__ CopyPools pools, const PageTable t, void* workspace,
                      int remap, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the plan
    const Workspace w = carve(workspace, t.n_pages);
    const int n_copies = *w.n_copies;
    if (WHOLE && remap) {
        const int total = t.batch * t.max_pages;
        for (long long i = blockIdx.x * (long long)kCopyThreads + threadIdx.x; i < total;
             i += gridDim.x * (long long)kCopyThreads) {
            const int page = t.table[i];
            if (page < 0) continue;
            const int to = page < t.n_pages ? w.list[page] : -1;
            if (to < 0) report(err, GEMMA_DEVERR_PAGE);  // no such page, or a free one
            else if (to != page) t.table[i] = to;
        }
    }
    const int per_copy = pools.unit0[pools.n];
    const long long units = (long long)n_copies * per_copy;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int ci = (int)(u / per_copy), r = (int)(u - (long long)ci * per_copy);
        int lo = 0, hi = pools.n - 1;  // the last pool whose units start at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (pools.unit0[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        const int4 c = w.copies[ci];
        const int row_bytes = pools.row_bytes[lo];
        const size_t head = (size_t)t.page_size * row_bytes, page = head * pools.n_kv[lo];
        const int in_pool = r - pools.unit0[lo];
        size_t off;
        long long left;
        if (WHOLE) {
            off = (size_t)in_pool * kCopyBytes;
            left = (long long)page - (long long)off;
        } else {
            const int per_head = (int)((head + kCopyBytes - 1) / kCopyBytes);
            const int h = in_pool / per_head;
            const size_t in_head = (size_t)(in_pool - h * per_head) * kCopyBytes;
            off = h * head + in_head;
            left = (long long)c.z * row_bytes - (long long)in_head;
        }
        if (left <= 0) continue;
        copy_span(pools.pool[lo] + c.y * page + off, pools.pool[lo] + c.x * page + off,
                  (int)(left < kCopyBytes ? left : kCopyBytes));
    }
}

template <bool WHOLE>
static cudaError_t launch_copies(const PagePools& pools, const PageTable& t, void* workspace,
                                 uint32_t* err, int n_sm, cudaStream_t st) {
    for (int p0 = 0; p0 < pools.n_pools; p0 += kPoolsPerLaunch) {
        CopyPools a = {};
        a.n = pools.n_pools - p0 < kPoolsPerLaunch ? pools.n_pools - p0 : kPoolsPerLaunch;
        for (int i = 0; i < a.n; ++i) {
            a.pool[i] = static_cast<uint8_t*>(pools.pools[p0 + i]);
            a.n_kv[i] = pools.n_kv[p0 + i];
            a.row_bytes[i] = pools.row_bytes[p0 + i];
            const size_t head = (size_t)t.page_size * a.row_bytes[i];
            const size_t units = WHOLE ? (head * a.n_kv[i] + kCopyBytes - 1) / kCopyBytes
                                       : (head + kCopyBytes - 1) / kCopyBytes * a.n_kv[i];
            if (a.unit0[i] + units > INT_MAX) return cudaErrorInvalidValue;
            a.unit0[i + 1] = a.unit0[i] + (int)units;
        }
        const cudaError_t e = launch_pdl(pages_copy_kernel<WHOLE>, dim3((unsigned)(4 * n_sm)),
                                         dim3(kCopyThreads), 0, st, a, t, workspace,
                                         (int)(p0 == 0), err);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// ---------------------------------------------------------------------------------------------
// reserve: private pages for positions [len, len + n_add) of every sequence
// ---------------------------------------------------------------------------------------------
// Items are the pages that a sequence is about to write, in the order of (sequence, position). A
// group of G threads (a power of two that fits the longest sequence's items) serves a sequence, each
// thread a run of consecutive items, so that thread order is item order within a stride of
// sequences. Shared pages: an item on one is marked in the table (-2 - page) while nothing else
// changes; then every marked item takes its reference off the page and enters its number into the
// page's minimum; what is left on the count are holders outside of the call, and where there are
// none the minimum's item keeps the page (a second mark, until nobody reads the count any more). The
// others, and items without a page, get the free pages in order.
__global__ void __launch_bounds__(kPlanThreads)
    pages_reserve_kernel(const PageTable t, const int32_t* __restrict__ seq_lens,
                         const int32_t* __restrict__ n_add, void* workspace, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    __shared__ int s_warp[32], s_max, s_copies;
    const Workspace w = carve(workspace, t.n_pages);
    const int tid = threadIdx.x;
    const long long cap = (long long)t.max_pages * t.page_size;

    // a sequence's items: blocks [blk0, blk1)
    auto items = [&](int b, int& blk0, int& blk1, int& len) -> bool {
        len = __ldg(seq_lens + b);
        const int add = __ldg(n_add + b);
        blk0 = blk1 = 0;
        if (len < 0 || add < 0 || (long long)len + add > cap) return false;
        if (add == 0) return true;
        blk0 = len / t.page_size;
        blk1 = (int)(((long long)len + add - 1) / t.page_size) + 1;
        return true;
    };
    if (tid == 0) s_max = 1, s_copies = 0;
    __syncthreads();
    int most = 0;
    for (int b = tid; b < t.batch; b += kPlanThreads) {
        int blk0, blk1, len;
        if (!items(b, blk0, blk1, len)) report(err, GEMMA_DEVERR_WRITE_POS);
        most = max(most, blk1 - blk0);
    }
    atomicMax(&s_max, most);
    __syncthreads();
    int G = 1;
    while (G < 32 && G < s_max) G *= 2;
    const int sub = tid & (G - 1), stride = kPlanThreads / G;
    // calls f(item's place in the table, its position's rows below len) for this thread's items of
    // the sequences b0 + tid / G
    auto each = [&](int b0, auto f) {
        const int b = b0 + tid / G;
        if (b >= t.batch) return;
        int blk0, blk1, len;
        items(b, blk0, blk1, len);
        const int q = (blk1 - blk0 + G - 1) / G;
        const int from = blk0 + sub * q, to = min(blk1, from + q);
        for (int blk = from; blk < to; ++blk)
            f(b * t.max_pages + blk, min(t.page_size, max(0, len - blk * t.page_size)));
    };

    // marks
    bool shared = false;
    for (int b0 = 0; b0 < t.batch; b0 += stride)
        each(b0, [&](int at, int) {
            const int page = t.table[at];
            if (page < -1) t.table[at] = -1;
            if (page < 0) return;
            if (page >= t.n_pages || t.refs[page] < 1) {
                report(err, GEMMA_DEVERR_PAGE);
            } else if (t.refs[page] > 1) {
                w.first[page] = INT_MAX;
                t.table[at] = -2 - page;
                shared = true;
            }
        });
    const bool any_shared = __syncthreads_or(shared);
    if (any_shared) {
        for (int b0 = 0; b0 < t.batch; b0 += stride)
            each(b0, [&](int at, int) {
                const int page = -2 - t.table[at];
                if (page < 0 || page >= t.n_pages) return;
                atomicSub(t.refs + page, 1);
                atomicMin(w.first + page, at);
            });
        __syncthreads();
        for (int b0 = 0; b0 < t.batch; b0 += stride)
            each(b0, [&](int at, int) {
                const int page = -2 - t.table[at];
                if (page < 0 || page >= t.n_pages) return;
                const int others = __ldcg(t.refs + page);
                if (others < 0) report(err, GEMMA_DEVERR_PAGE);
                if (others <= 0 && __ldcg(w.first + page) == at) t.table[at] = -2 - page - kKeeper;
            });
        __syncthreads();
    }
    // the pages needed in all (keepers take their reference back)
    int need = 0;
    for (int b0 = 0; b0 < t.batch; b0 += stride)
        each(b0, [&](int at, int) {
            const int e = t.table[at];
            if (e < -1 - kKeeper) {
                const int page = -2 - kKeeper - e;
                t.table[at] = page;
                if (page < t.n_pages) t.refs[page] = 1;
            } else if (e < 0) {
                ++need;
            }
        });
    int total = 0;
    block_scan(need, s_warp, &total);
    // the first `total` free pages
    int n_free = 0;
    for (int p0 = 0; p0 < t.n_pages && n_free < total; p0 += 4 * kPlanThreads) {
        const int at = p0 + 4 * tid;
        bool is_free[4];
        int mine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            is_free[j] = at + j < t.n_pages && __ldcg(t.refs + at + j) == 0;
            mine += is_free[j];
        }
        int found = 0;
        int k = n_free + block_scan(mine, s_warp, &found);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (is_free[j]) {
                if (k < total) w.list[k] = at + j;
                ++k;
            }
        n_free += found;
    }
    __syncthreads();
    n_free = min(n_free, total);
    // given out in order
    int given = 0;
    for (int b0 = 0; b0 < t.batch && total > 0; b0 += stride) {
        int mine = 0, sum = 0;
        each(b0, [&](int at, int) { mine += t.table[at] < 0; });
        int k = given + block_scan(mine, s_warp, &sum);
        given += sum;
        each(b0, [&](int at, int rows) {
            const int e = t.table[at];
            if (e >= 0) return;
            const int old = -2 - e < t.n_pages ? -2 - e : -1;
            if (k < n_free) {
                const int page = w.list[k];
                t.table[at] = page;
                t.refs[page] = 1;
                if (old >= 0 && rows > 0)
                    w.copies[atomicAdd(&s_copies, 1)] = make_int4(old, page, rows, 0);
            } else {
                report(err, GEMMA_DEVERR_POOL_FULL);
                if (old >= 0) {  // stays shared
                    t.table[at] = old;
                    atomicAdd(t.refs + old, 1);
                }
            }
            ++k;
        });
    }
    __syncthreads();
    if (tid == 0) *w.n_copies = s_copies;
}

cudaError_t launch_pages_reserve(const PagePools& pools, const PageTable& t,
                                 const int32_t* seq_lens, const int32_t* n_add, void* workspace,
                                 uint32_t* err, int n_sm, cudaStream_t st) {
    const cudaError_t e = launch_pdl(pages_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, st, t,
                                     seq_lens, n_add, workspace, err);
    return e == cudaSuccess ? launch_copies<false>(pools, t, workspace, err, n_sm, st) : e;
}

// ---------------------------------------------------------------------------------------------
// compact: the i-th used page at or behind n_used moves to the i-th free page before it
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads)
    pages_compact_kernel(const PageTable t, int32_t* n_used_out, void* workspace, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    __shared__ int s_warp[32], s_below;
    const Workspace w = carve(workspace, t.n_pages);
    const int tid = threadIdx.x;
    // thread tid looks at the pages [p0, p1)
    const int per = (t.n_pages + kPlanThreads - 1) / kPlanThreads;
    const int p0 = min((long long)t.n_pages, (long long)tid * per), p1 = min(t.n_pages, p0 + per);
    // (the counts are read once, so that what follows agrees with itself whatever they hold)
    int mine = 0, n_used = 0;
#pragma unroll 4
    for (int p = p0; p < p1; ++p) {
        const int used = t.refs[p] > 0;
        w.list[p] = used;
        mine += used;
    }
    const int before = block_scan(mine, s_warp, &n_used);
    // used pages among the first n_used
    if (n_used >= p0 && (n_used < p1 || (tid == kPlanThreads - 1 && n_used == t.n_pages))) {
        int k = before;
        for (int p = p0; p < n_used; ++p) k += w.list[p];
        s_below = k;
    }
    __syncthreads();
    const int below = s_below, moves = n_used - below;
    int k = before;
    for (int p = p0; p < p1; ++p) {
        const int used = w.list[p];
        if (p < n_used) {
            if (!used) w.first[p - k] = p;  // a hole
            w.list[p] = used ? p : -1;
        } else {
            if (used) w.spare[k - below] = p;  // a page to move
            w.list[p] = -1;
        }
        k += used;
    }
    __syncthreads();
    for (int i = tid; i < moves; i += kPlanThreads) {
        const int from = w.spare[i], to = w.first[i];
        w.copies[i] = make_int4(from, to, t.page_size, 0);
        w.list[from] = to;
        t.refs[to] = t.refs[from];
        t.refs[from] = 0;
    }
    if (tid == 0) {
        *w.n_copies = moves;
        if (n_used_out) *n_used_out = n_used;
    }
}

cudaError_t launch_pages_compact(const PagePools& pools, const PageTable& t, int32_t* n_used,
                                 void* workspace, uint32_t* err, int n_sm, cudaStream_t st) {
    const cudaError_t e = launch_pdl(pages_compact_kernel, dim3(1), dim3(kPlanThreads), 0, st, t,
                                     n_used, workspace, err);
    return e == cudaSuccess ? launch_copies<true>(pools, t, workspace, err, n_sm, st) : e;
}

}  // namespace gemma
