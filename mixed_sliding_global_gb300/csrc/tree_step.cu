// tree_step.cu -- what follows the verification of a drafted tree: the accepted path, and the move
// of its rows to where the sequence goes on, in every cache.
#include "common.cuh"
#include "tree.h"

namespace gemma {

// ---------------------------------------------------------------------------------------------
// accept: from the root, on to the lowest child whose token is the one drawn behind the node
// ---------------------------------------------------------------------------------------------
// One warp per sequence, node lane + 32 k in register k. A step of the walk is a ballot per
// register; children have higher indices than their parent, so it takes at most n steps.
constexpr int kAcceptWarps = 4;
constexpr int kNodeRegs = kTreeMaxNodes / 32;

__global__ void __launch_bounds__(kAcceptWarps * 32)
    tree_accept_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ parents,
                       const int32_t* __restrict__ next, const int32_t* __restrict__ n_real,
                       const int32_t* seq_lens, int batch, int n, int32_t* __restrict__ path,
                       int32_t* __restrict__ n_keep, int32_t* __restrict__ token,
                       int32_t* lens_out, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
    if (b >= batch) return;
    const size_t row = (size_t)b * n;
    // (the whole bucket, so that nothing waits for n_real)
    int tok[kNodeRegs], par[kNodeRegs], nxt[kNodeRegs], out[kNodeRegs];
#pragma unroll
    for (int k = 0; k < kNodeRegs; ++k) {
        const int i = lane + 32 * k;
        tok[k] = i < n ? __ldg(tokens + row + i) : -1;
        par[k] = i < n ? __ldg(parents + row + i) : -1;
        nxt[k] = i < n ? __ldg(next + row + i) : -1;
        out[k] = -1;
    }
    const int nr = n_real ? __ldg(n_real + b) : n;
    const int len = seq_lens ? seq_lens[b] : 0;
    const bool bad_real = nr < 0 || nr > n;
    const bool bad_len = !bad_real && seq_lens && len < nr;
    bool bad_node = false;
#pragma unroll
    for (int k = 0; k < kNodeRegs; ++k) {
        const int i = lane + 32 * k;
        const bool live = !bad_real && i < nr;
        if (!live) tok[k] = par[k] = nxt[k] = -1;
        bad_node |= live && (par[k] < -1 || par[k] >= i);
    }
    const bool bad_tree = __any_sync(0xffffffffu, bad_node);
    int cnt = 0, last = -1;
    if (!bad_real && !bad_len && !bad_tree && nr > 0) {
        int cur = 0;
        for (;;) {
            if (lane == (cnt & 31)) {
#pragma unroll
                for (int k = 0; k < kNodeRegs; ++k)
                    if (k == cnt >> 5) out[k] = cur;
            }
            ++cnt;
            int mine = nxt[0];
#pragma unroll
            for (int k = 1; k < kNodeRegs; ++k) mine = cur >> 5 == k ? nxt[k] : mine;
            last = __shfl_sync(0xffffffffu, mine, cur & 31);
            int child = -1;
#pragma unroll
            for (int k = kNodeRegs - 1; k >= 0; --k) {
                // (a node that is not there has parent -1, which no current node is)
                const unsigned hit =
                    __ballot_sync(0xffffffffu, par[k] == cur && tok[k] == last && last >= 0);
                if (hit) child = 32 * k + __ffs(hit) - 1;
            }
            if (child < 0) break;
            cur = child;
        }
    }
#pragma unroll
    for (int k = 0; k < kNodeRegs; ++k)
        if (lane + 32 * k < n) path[row + lane + 32 * k] = out[k];
    if (lane == 0) {
        n_keep[b] = cnt;
        token[b] = last;
        if (lens_out) lens_out[b] = bad_real || bad_len ? len : len - nr + cnt;
        if (bad_real) report(err, GEMMA_DEVERR_N_REAL);
        else if (bad_len) report(err, GEMMA_DEVERR_SEQ_LEN);
        else if (bad_tree) report(err, GEMMA_DEVERR_TREE);
    }
}

cudaError_t launch_tree_accept(const int32_t* tokens, const int32_t* parents, const int32_t* next,
                               const int32_t* n_real, const int32_t* seq_lens, int batch, int n,
                               int32_t* path, int32_t* n_keep, int32_t* token, int32_t* lens_out,
                               uint32_t* err, cudaStream_t st) {
    return launch_pdl(tree_accept_kernel, dim3((unsigned)((batch + kAcceptWarps - 1) / kAcceptWarps)),
                      dim3(kAcceptWarps * 32), 0, st, tokens, parents, next, n_real, seq_lens,
                      batch, n, path, n_keep, token, lens_out, err);
}

// ---------------------------------------------------------------------------------------------
// keep: row base + i := row base + path[i], i < n_keep, in every cache of the call
// ---------------------------------------------------------------------------------------------
// A thread moves one vector column of the rows of one head of one cache, so no two threads touch
// the same bytes and the order of a thread's own loads and stores is all that counts. path rises
// strictly, so path[i] >= i: the rows a batch of kKeepBatch stores overwrites are sources of that
// batch (loaded before) or of earlier ones, never of later ones.
constexpr int kKeepThreads = 256;
constexpr int kKeepBatch = 8;
constexpr int kKeepCaches = 128;  // cache pointers per launch (kernel arguments)

struct KeepPtrs {
    uint8_t* p[kKeepCaches];
};

template <typename V>
__global__ void __launch_bounds__(kKeepThreads)
    kv_keep_kernel(const __grid_constant__ KeepPtrs caches, const KeepLayout k, uint32_t* err) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    __shared__ long long s_row[kTreeMaxNodes];  // row of position base + i (head 0), -1: no page
    __shared__ int s_path[kTreeMaxNodes];
    const int b = blockIdx.z, tid = threadIdx.x;
    const int nk = __ldg(k.n_keep + b);
    const int pos = __ldg(k.write_pos + b);
    // (of the whole bucket, so that it does not wait for n_keep)
    const int m = tid < k.n ? __ldg(k.path + (size_t)b * k.n + tid) : 0;
    const int before = tid && tid < k.n ? __ldg(k.path + (size_t)b * k.n + tid - 1) : -1;
    const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
    if (nk < 0 || nk > k.n) {
        if (first_cta && tid == 0) report(err, GEMMA_DEVERR_TREE);
        return;
    }
    if (nk == 0) return;
    bool bad = false, move = false;
    if (tid < nk) {
        bad = m <= before || m >= k.n;
        move = m != tid;
        s_path[tid] = m;
    }
    const bool bad_path = __syncthreads_or(bad);
    const int identity = nk - __syncthreads_count(move);  // leading rows that stay where they are
    if (bad_path) {
        if (first_cta && tid == 0) report(err, GEMMA_DEVERR_TREE);
        return;
    }
    const int last = s_path[nk - 1];
    if (pos < 0 || (!k.ring && (long long)pos + last >= k.cap)) {
        if (first_cta && tid == 0) report(err, GEMMA_DEVERR_WRITE_POS);
        return;
    }
    if (identity == nk) return;
    const int slots = k.pg.block_table ? k.pg.page_size : k.cap;
    if (tid <= last) {
        long long row;
        if (k.pg.block_table) {
            const int at = pos + tid, blk = at / k.pg.page_size;
            const int page = __ldg(k.pg.block_table + (size_t)b * k.pg.max_pages + blk);
            row = (long long)page * k.n_kv * slots + (at - blk * k.pg.page_size);
            if (page < 0 || page >= k.pg.n_pages) row = -1;
        } else {
            const long long at = (long long)pos + tid;
            row = (long long)b * k.n_kv * slots + (k.ring ? at % k.ring : at);
        }
        s_row[tid] = row;
    }
    __syncthreads();
    const int vecs = k.row_bytes / (int)sizeof(V);
    const int col = blockIdx.x * kKeepThreads + tid;
    const int h = col / vecs;
    if (h >= k.n_kv) return;
    V* cache = reinterpret_cast<V*>(caches.p[blockIdx.y]) + (size_t)h * slots * vecs +
               (col - h * vecs);
    bool lost = false;
    for (int i0 = identity; i0 < nk; i0 += kKeepBatch) {
        V v[kKeepBatch];
        bool have[kKeepBatch];
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j) {
            const int i = i0 + j;
            have[j] = false;
            if (i < nk) {
                const long long from = s_row[s_path[i]];
                have[j] = from >= 0 && s_row[i] >= 0;
                if (have[j]) v[j] = cache[(size_t)from * vecs];
                else lost = true;
            }
        }
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j)
            if (have[j]) cache[(size_t)s_row[i0 + j] * vecs] = v[j];
    }
    if (lost) report(err, GEMMA_DEVERR_PAGE);
}

cudaError_t launch_kv_keep(void* const* caches, int n_caches, const KeepLayout& k, int batch,
                           uint32_t* err, cudaStream_t st) {
    const int width = k.row_bytes % 16 == 0  ? 16
                      : k.row_bytes % 8 == 0 ? 8
                      : k.row_bytes % 4 == 0 ? 4
                                             : 2;
    const long long cols = (long long)k.n_kv * (k.row_bytes / width);
    for (int c0 = 0; c0 < n_caches; c0 += kKeepCaches) {
        const int n = n_caches - c0 < kKeepCaches ? n_caches - c0 : kKeepCaches;
        KeepPtrs ptrs = {};
        for (int i = 0; i < n; ++i) ptrs.p[i] = static_cast<uint8_t*>(caches[c0 + i]);
        const dim3 grid((unsigned)((cols + kKeepThreads - 1) / kKeepThreads), n, batch);
        const dim3 block(kKeepThreads);
        const cudaError_t e =
            width == 16  ? launch_pdl(kv_keep_kernel<uint4>, grid, block, 0, st, ptrs, k, err)
            : width == 8 ? launch_pdl(kv_keep_kernel<uint2>, grid, block, 0, st, ptrs, k, err)
            : width == 4 ? launch_pdl(kv_keep_kernel<uint32_t>, grid, block, 0, st, ptrs, k, err)
                         : launch_pdl(kv_keep_kernel<uint16_t>, grid, block, 0, st, ptrs, k, err);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gemma
