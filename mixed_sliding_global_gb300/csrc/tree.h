// tree.h -- launch interfaces of the drafted-tree step and of the page bookkeeping (api.cu).
#pragma once

#include "attn_internal.h"

namespace gemma {

constexpr int kTreeMaxNodes = 128;  // nodes of a tree: an ancestor set is four words
constexpr int kTreeKeyTile = 64;    // keys per tile; chunks of keys are multiples of it

// One attention launch over trees. p: n_tok = nodes of the bucket, n_real the sequences' own
// (nullptr: all); o_part [batch][n_kv][rows][n_split][D] and ml_part [..][n_split][2] hold the
// partial results of n_split > 1 chunks of p.chunk keys (rows = nodes x G).
struct TreeParams {
    RowsParams p;
    const int32_t* parents;  // [batch][n_tok], -1 or an earlier node
    int n_sm;                // of the device
};

constexpr int kTreeRowsMax = 32;  // rows per KV head of launch_tree_rows

// How units (a KV head of a sequence and a tile of rows) are dealt out to workers: in equal shares of their
// key tiles, parts merged; each to a pair or cluster of its own; or whole ones in about equal shares. Only
// the first needs a workspace.
enum { kTreeShares, kTreeAlone, kTreeWhole };

// On CTA pairs (tree_pair.cu), head_dim 256 and 512, any number of rows; the merge included. workers:
// pairs, one per two SMs at most, or, alone, one per unit.
size_t tree_pair_workspace(int batch, int workers);
cudaError_t launch_tree_pair(const TreeParams& tp, int head_dim, int batch, void* workspace,
                             int workers, int deal, cudaStream_t st);
// On single SMs with tcgen05 (tree_tc.cu), head_dim 64 to 256, any number of rows; the merge included.
// workers: CTAs, one per SM at most; or a cluster of 1 to 8 CTAs for each unit (cluster > 0; no workspace).
int tree_tc_clusters(int head_dim, int cluster);  // clusters of 2, 4 or 8 that run at once
size_t tree_tc_workspace(int head_dim, int batch, int workers);
cudaError_t launch_tree_tc(const TreeParams& tp, int head_dim, int batch, void* workspace,
                           int workers, int cluster, int deal, cudaStream_t st);

// Parts of units cut into equal shares of the key tiles, and where they lie in the workspace. A worker
// has two slots: for the part that its share begins with, and for the one that it ends with.
struct MergeParams {
    TreeParams tp;
    int batch, n_rt;  // row tiles per (sequence, KV head)
    int workers;      // (CTAs of a unit's cluster where units are dealt out by the host)
    int keys;         // of a key tile
    float* part_o;    // [2 workers][pieces of 128 rows and up to 256 columns][columns / 4][128][4]
    float2* part_ml;  // [2 workers][pieces][128]
    int32_t* before;  // [batch + 1] key tiles of earlier sequences; then whether no unit was cut
};
cudaError_t launch_tree_merge(const MergeParams& mp, int head_dim, int rows, cudaStream_t st);

// On mma.sync (tree_attn.cu): head_dim 64 and 128 with up to 16 rows, 512 with up to 32; the CTAs that fit
// an SM.
int tree_ctas_per_sm(int head_dim);
cudaError_t launch_tree_rows(const TreeParams& tp, int head_dim, int batch, cudaStream_t st);
cudaError_t launch_tree_f32(const TreeParams& tp, int head_dim, int batch, cudaStream_t st);
cudaError_t launch_tree_combine(const TreeParams& tp, int head_dim, int batch, cudaStream_t st);

cudaError_t launch_tree_accept(const int32_t* tokens, const int32_t* parents, const int32_t* next,
                               const int32_t* n_real, const int32_t* seq_lens, int batch, int n,
                               int32_t* path, int32_t* n_keep, int32_t* token, int32_t* lens_out,
                               uint32_t* err, cudaStream_t st);

// Rows of row_bytes bytes in caches [batch][n_kv][cap] or pools [n_pages][n_kv][page_size].
struct KeepLayout {
    const int32_t* write_pos;
    const int32_t* path;
    const int32_t* n_keep;
    PagedLayout pg;
    int n, n_kv, cap, ring;
    int row_bytes;
};
cudaError_t launch_kv_keep(void* const* caches, int n_caches, const KeepLayout& k, int batch,
                           uint32_t* err, cudaStream_t st);

// Pools that share a block table and page numbers.
struct PagePools {
    void* const* pools;
    const int32_t* n_kv;
    const int32_t* row_bytes;
    int n_pools;
};
// A block table and the reference counts of its pages.
struct PageTable {
    int32_t* table;  // [batch][max_pages]
    int32_t* refs;   // [n_pages]
    int max_pages, page_size, n_pages, batch;
};
constexpr int kMaxPages = 1 << 29;  // of a pool whose pages are moved or given out
constexpr size_t pages_workspace(int n_pages) { return 256 + 28 * ((size_t)n_pages + 4); }
cudaError_t launch_pages_free(const PageTable& t, const int32_t* keep_from, const int32_t* keep_to,
                              uint32_t* err, int n_sm, cudaStream_t st);
cudaError_t launch_pages_fork(const PageTable& t, int32_t* seq_lens, const int32_t* src,
                              const int32_t* dst, int n, uint32_t* err, cudaStream_t st);
cudaError_t launch_pages_reserve(const PagePools& pools, const PageTable& t,
                                 const int32_t* seq_lens, const int32_t* n_add, void* workspace,
                                 uint32_t* err, int n_sm, cudaStream_t st);
cudaError_t launch_pages_compact(const PagePools& pools, const PageTable& t, int32_t* n_used,
                                 void* workspace, uint32_t* err, int n_sm, cudaStream_t st);

}  // namespace gemma
